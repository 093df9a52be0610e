"""What the rotary and cache entry points refuse, before anything is enqueued (CPU): the C
calls get pointers that are never followed."""

import ctypes

import pytest
import torch

import post_weight_quantization_act_amd as awq

INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3
P = 1 << 20     # an aligned address nothing reads


def strides(*v):
    return (ctypes.c_int64 * len(v))(*v)


def cache(**over):
    f = dict(k_codes=P, v_codes=P, k_steps=P, v_steps=P, n_pages=4, kv_heads=2, head_dim=64, page=16)
    f.update(over)
    return ctypes.addressof(hold(awq.KvCacheStruct(**f)))


_held = []


def hold(x):
    _held.append(x)
    return x


def status(fn, args):
    got = getattr(awq.library(), fn)(*args.values())
    if got != 0:
        assert awq.library().awq_last_error()
    return got


def table_args(**over):
    a = dict(n_pos=8, rot=64, base=1e4, scaling=None, table=P, stream=None)
    a.update(over)
    return a


@pytest.mark.parametrize("over,want", [
    (dict(n_pos=0), INVALID), (dict(rot=0), INVALID), (dict(rot=7), INVALID),
    (dict(base=0.0), INVALID), (dict(base=float("inf")), INVALID), (dict(base=float("nan")), INVALID),
    (dict(table=None), INVALID), (dict(table=P + 4), UNSUPPORTED), (dict(n_pos=1 << 40), UNSUPPORTED),
    (dict(scaling=(9, 1, 1, 1, 2, 1)), INVALID), (dict(scaling=(1, 0, 1, 1, 2, 1)), INVALID),
    (dict(scaling=(2, 1, 0, 1, 2, 1)), INVALID), (dict(scaling=(2, 1, 1, 2, 2, 1)), INVALID),
    (dict(scaling=(3, 1, 1, 0, 2, 1)), INVALID), (dict(scaling=(0, 1, 1, 1, 2, float("nan"))), INVALID),
])
def test_rope_table_refuses(over, want):
    if "scaling" in over:
        over = dict(scaling=ctypes.byref(awq.RopeScaling(*over["scaling"])))
    assert status("awq_rope_table", table_args(**over)) == want


def rope_args(**over):
    a = dict(x=P, x_dtype=1, B=1, S=2, H=3, D=64, xs=strides(384, 192, 64), positions=None, pst=0,
             table=P, n_pos=8, rot=64, flags=0, out=P, out_dtype=1, os=strides(384, 192, 64),
             stream=None)
    a.update(over)
    return a


@pytest.mark.parametrize("over,want", [
    (dict(x_dtype=7), INVALID), (dict(out_dtype=-1), INVALID), (dict(B=-1), INVALID),
    (dict(D=0), INVALID), (dict(flags=4), INVALID), (dict(rot=0), INVALID), (dict(rot=3), INVALID),
    (dict(rot=66), INVALID), (dict(n_pos=0), INVALID), (dict(x=None), INVALID),
    (dict(out=None), INVALID), (dict(table=None), INVALID), (dict(xs=None), INVALID),
    (dict(x=P + 1), UNSUPPORTED), (dict(positions=P + 2), UNSUPPORTED),
    (dict(D=65538), UNSUPPORTED), (dict(B=1 << 31), UNSUPPORTED),
    (dict(B=1 << 20, S=1 << 20), UNSUPPORTED), (dict(S=0), 0),
])
def test_rope_refuses(over, want):
    assert status("awq_rope", rope_args(**over)) == want


def append_args(**over):
    a = dict(cache=cache(), k=P, v=P, dtype=1, T=3, st=strides(128, 64, 128, 64), starts=P, lens=P,
             B=2, pages=P, max_pages=4, max_new=3, table=P, n_pos=8, rot=64, flags=0,
             positions=None, q=P, Hq=4, qs=strides(256, 64), q_out=P, q_dtype=2, stream=None)
    a.update(over)
    return a


CACHE_REFUSALS = [
    (dict(cache=None), INVALID), (dict(cache=dict(kv_heads=0)), INVALID),
    (dict(cache=dict(n_pages=0)), INVALID), (dict(cache=dict(head_dim=60)), UNSUPPORTED),
    (dict(cache=dict(head_dim=264)), UNSUPPORTED), (dict(cache=dict(page=24)), UNSUPPORTED),
    (dict(cache=dict(page=8)), UNSUPPORTED), (dict(cache=dict(page=512)), UNSUPPORTED),
    (dict(cache=dict(n_pages=1 << 31)), UNSUPPORTED), (dict(cache=dict(k_codes=None)), INVALID),
    (dict(cache=dict(v_codes=P + 8)), UNSUPPORTED), (dict(cache=dict(k_steps=P + 2)), UNSUPPORTED),
    (dict(T=-1), INVALID), (dict(max_pages=-1), INVALID), (dict(starts=None), INVALID),
    (dict(pages=None), INVALID), (dict(max_new=0), INVALID), (dict(max_pages=0), INVALID),
    (dict(T=1 << 31), UNSUPPORTED), (dict(pages=P + 1), UNSUPPORTED), (dict(starts=P + 1), UNSUPPORTED),
    (dict(B=1 << 31), UNSUPPORTED), (dict(B=0), 0), (dict(T=0), 0),
]


def built(args, over):
    over = dict(over)
    if isinstance(over.get("cache"), dict):
        over["cache"] = cache(**over["cache"])
    return args(**over)


@pytest.mark.parametrize("over,want", CACHE_REFUSALS + [
    (dict(dtype=3), INVALID), (dict(q_dtype=3), INVALID), (dict(flags=2), INVALID),
    (dict(rot=66), INVALID), (dict(rot=1), INVALID), (dict(n_pos=0), INVALID),
    (dict(table=None), INVALID), (dict(Hq=3), INVALID), (dict(q=None), INVALID),
    (dict(q_out=None), INVALID), (dict(qs=None), INVALID), (dict(k=None), INVALID),
    (dict(st=None), INVALID), (dict(lens=None), INVALID), (dict(k=P + 1), UNSUPPORTED),
    (dict(q_out=P + 8), UNSUPPORTED),
])
def test_append_refuses(over, want):
    assert status("awq_kv_append", built(append_args, over)) == want


def read_args(**over):
    a = dict(cache=cache(), T=3, starts=P, first=P, B=2, pages=P, max_pages=4, max_new=3, k=P, v=P,
             dtype=0, stream=None)
    a.update(over)
    return a


@pytest.mark.parametrize("over,want", CACHE_REFUSALS + [
    (dict(dtype=3), INVALID), (dict(first=None), INVALID), (dict(k=None), INVALID),
    (dict(v=P + 8), UNSUPPORTED),
])
def test_read_refuses(over, want):
    assert status("awq_kv_read", built(read_args, over)) == want


def attention_args(**over):
    a = dict(cache=cache(), q=P, dtype=1, T=3, Hq=4, qs=strides(256, 64), starts=P, lens=P, B=2,
             pages=P, max_pages=4096, max_new=3, max_len=65536, scale=0.125, window=0, flags=0, out=P,
             lse=None, ws=P, ws_bytes=1 << 40, stream=None)
    a.update(over)
    return a


@pytest.mark.parametrize("over,want", CACHE_REFUSALS + [
    (dict(dtype=3), INVALID), (dict(dtype=0), UNSUPPORTED), (dict(Hq=3), INVALID),
    (dict(Hq=0), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=-1.0), INVALID),
    (dict(scale=1e300), INVALID), (dict(window=-1), INVALID), (dict(max_len=-1), INVALID),
    (dict(flags=2), INVALID), (dict(q=None), INVALID), (dict(qs=None), INVALID),
    (dict(lens=None), INVALID), (dict(out=None), INVALID), (dict(out=P + 4), UNSUPPORTED),
    (dict(q=P + 1), UNSUPPORTED),
])
def test_attention_refuses(over, want):
    assert status("awq_kv_attention", built(attention_args, over)) == want


def test_binding_refuses():
    x = torch.zeros(2, 3, 64)
    table = torch.zeros(4, 32, 2)
    with pytest.raises(ValueError, match="GPU tensor"):
        awq.awq_rope(x, table)
    with pytest.raises(TypeError):
        awq.awq_rope([1.0], table)
    with pytest.raises(ValueError, match="scaling"):
        awq.awq_rope_table(4, 64, scaling="no such")
    with pytest.raises(ValueError, match="GPU tensor"):
        awq.KvCache.empty(2, 1, 16, 64, device="cpu")
    for call in (awq.awq_kv_append, awq.awq_kv_attention):
        with pytest.raises(TypeError, match="KvCache"):
            call(None, x, x, x, x)
    with pytest.raises(TypeError, match="KvCache"):
        awq.awq_kv_read(None, x, x)


def test_attention_workspace_size_is_host_only_and_bounded():
    size = awq.awq_kv_attention_workspace_size
    assert size(0, 1, 8, 8, 128, 1, 100) == 0 and size(1, 1, 7, 2, 128, 1, 100) == 0
    assert size(64, 64, 64, 8, 128, 1, 8192) < 1 << 30
    assert size(1, 1, 64, 8, 128, 1, 1 << 20) < 1 << 28
