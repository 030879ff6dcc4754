"""Serving calls without tokens or rows do nothing and succeed: an empty tensor has no address (no GPU needed)."""
import pytest

from test_serving_args import APPEND, APPEND_ARGS, ATTN, ATTN_ARGS, PTR, call, lib  # noqa: F401


@pytest.mark.parametrize("name,types,args", [("dspark_kv_append", APPEND, APPEND_ARGS), ("dspark_prefix_attention", ATTN, ATTN_ARGS)])
def test_no_tokens_is_no_error(lib, name, types, args):  # noqa: F811
    nothing = {n: None if t is PTR and n != "ws" else args[n] for n, t in types}
    assert call(lib, name, types, nothing, T=0) == 0
    # of an empty step's tensors only those with a row a token are empty
    no_rows = {n: None if n in ("q", "k", "v", "slots", "out", "lse") and t is PTR else args[n] for n, t in types}
    assert call(lib, name, types, no_rows, T=0) == 0
