"""Tensors of two devices in one call are refused before anything else (on the
CPU: fake tensors carry a device and nothing behind it)."""
import pytest

from helpers import ensure_lib

torch = pytest.importorskip("torch")
fake_tensor = pytest.importorskip("torch._subclasses.fake_tensor")


def _calls(mx):
    """name -> (shape and type of every tensor argument, call)"""
    f32, b16, i32 = torch.float32, torch.bfloat16, torch.int32
    batch = dict(cu_q=((2,), i32), ctx_len=((1,), i32), page_table=((1, 4), i32))
    cache = dict(k_cache=((4, 2, 16, 64), b16), v_cache=((4, 2, 16, 64), b16))
    return {
        "add_rms_norm": (dict(x=((2, 64), f32), gamma=((64,), f32), residual=((2, 64), f32), sum_out=((2, 64), f32),
                              y=((2, 64), b16), q=((2, 64), torch.int8), ds=((2, 2, 2), f32)),
                         lambda **t: mx.add_rms_norm(quantize=True, **t)),
        "dequantize_q8_1": (dict(q=((2, 64), torch.int8), ds=((2, 2, 2), f32), y=((2, 64), f32)), mx.dequantize_q8_1),
        "route_experts": (dict(logits=((2, 64), f32), bias=((64,), f32), ids=((2, 4), i32), w=((2, 4), f32)),
                          lambda **t: mx.route_experts(k=4, **t)),
        "rope_kv_write": (dict(qkv=((3, 512), f32), cos_sin=((9, 64), f32), q=((3, 4, 64), b16), **cache, **batch),
                          lambda **t: mx.rope_kv_write(n_heads=4, **t)),
        "paged_attention": (dict(q=((3, 4, 64), b16), out=((3, 4, 64), b16), lse=((3, 4), f32),
                                 ws=((64,), torch.uint8), **cache, **batch), mx.paged_attention),
        "paged_attention_workspace_bytes": (dict(**cache, **batch),
                                            lambda **t: mx.paged_attention_workspace_bytes(n_tokens=3, n_heads=4, **t)),
    }


@pytest.mark.parametrize("name", ["add_rms_norm", "dequantize_q8_1", "route_experts", "rope_kv_write",
                                  "paged_attention", "paged_attention_workspace_bytes"])
def test_tensors_of_another_device_are_refused(name):
    import moe_expert_gb300 as mx
    ensure_lib()
    args, call = _calls(mx)[name]
    for odd in args:
        for where, say in (("cuda:1", "one device"), ("cpu", "CUDA|one device")):
            with fake_tensor.FakeTensorMode():
                t = {k: torch.empty(shape, dtype=dt, device=where if k == odd else "cuda:0")
                     for k, (shape, dt) in args.items()}
            with pytest.raises(ValueError, match=say):
                call(**t)
