"""What the rotary and cache entry points decide on the host, at the edges of their sizes (CPU): the
C calls get pointers that are never followed, and return before anything is enqueued."""

from test_kv_abi import UNSUPPORTED, rope_args, status, strides


def test_rope_refuses_rows_past_its_items():
    assert status("awq_rope", rope_args(B=1, S=1, H=1 << 20, D=65536, xs=strides(0, 0, 65536),
                                        os=strides(0, 0, 65536))) == UNSUPPORTED
