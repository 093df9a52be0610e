"""What the rotary and cache entry points decide on the host, at the edges of their sizes (CPU): the
C calls get pointers that are never followed, and return before anything is enqueued."""

from test_kv_abi import INVALID, UNSUPPORTED, append_args, rope_args, status, strides


def test_rope_refuses_rows_past_its_items():
    assert status("awq_rope", rope_args(B=1, S=1, H=1 << 20, D=65536, xs=strides(0, 0, 65536),
                                        os=strides(0, 0, 65536))) == UNSUPPORTED


def test_append_of_no_rows_takes_an_empty_q():
    """Torch's empty tensors have null pointers."""
    nothing = dict(T=0, k=None, v=None, q=None, q_out=None)
    assert status("awq_kv_append", append_args(**nothing)) == 0
    assert status("awq_kv_append", append_args(**nothing, B=0, starts=None, lens=None, pages=None)) == 0
    assert status("awq_kv_append", append_args(q=None)) == INVALID
