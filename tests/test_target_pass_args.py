"""What the calls after the target's pass refuse on the host, before anything touches the GPU (no GPU needed)."""
import pytest

from test_serving_args import F32, I32, INVALID, P, PTR, SIZE, WORKSPACE, call, lib  # noqa: F401

TAIL = [("ws", PTR), ("bytes", SIZE), ("stream", PTR)]


def spec(ints, *rest):
    return [(n, I32) for n in ints.split()] + [(n, F32 if n == "tau" else I32 if n in ("out_dtype",) else PTR) for n in
                                             " ".join(rest).split()] + TAIL


CALLS = {
    "dspark_probabilities": (spec("N V dtype", "logits temperature out_dtype probs"), {}, "logits temperature probs",
                             [dict(N=-1), dict(V=0), dict(V=(1 << 20) + 1), dict(dtype=2), dict(out_dtype=-1), dict(N=1 << 25)]),
    "dspark_verify_probs": (spec("R gamma V T dtype", "target q_start draft tokens u out accepted p_tok"), {},
                            "target q_start tokens u out accepted p_tok",
                            [dict(R=0), dict(gamma=0), dict(V=0), dict(V=(1 << 20) + 1), dict(T=-1), dict(dtype=3)]),
    "dspark_page_collect": (spec("R page max_pages n_pages n_pinned", "table kv_len pinned refs free n_free"), {},
                            "table kv_len pinned refs free n_free",
                            [dict(R=0), dict(page=0), dict(max_pages=0), dict(n_pages=0), dict(n_pinned=-1)]),
    "dspark_page_fork": (spec("R_from R page max_pages n_pages n_free n_pinned",
                              "table kv_len parent fork_len free pinned new_table new_len src dst tokens used"),
                         {"new_table": 2 * P}, "table kv_len parent free pinned new_table new_len src dst tokens used",
                         [dict(R_from=0), dict(R=0), dict(page=0), dict(max_pages=0), dict(n_pages=0), dict(n_free=-1),
                          dict(n_pinned=-1), dict(new_table=P), dict(page=1 << 16, max_pages=1 << 16)]),
    "dspark_page_compact": (spec("R page max_pages n_pages n_pinned", "table kv_len pinned new_table new_pinned src dst n_live"), {},
                            "table kv_len pinned new_table new_pinned src dst n_live",
                            [dict(R=0), dict(page=0), dict(max_pages=0), dict(n_pages=0), dict(n_pinned=-1)]),
    "dspark_page_copy": (spec("n layers n_pages page Hkv D dtype", "src dst tokens k_cache v_cache"), {}, "src dst k_cache v_cache",
                         [dict(n=-1), dict(layers=0), dict(n_pages=0), dict(page=0), dict(Hkv=0), dict(D=0), dict(dtype=9),
                          dict(Hkv=1 << 13, D=1 << 13), dict(page=1 << 20, Hkv=1 << 10, D=1 << 10)]),
    "dspark_distill": (spec("N V K dtype", "logits ids teacher lse weight tau loss grad"), {"tau": 1.0}, "logits ids teacher loss",
                       [dict(N=-1), dict(V=0), dict(V=(1 << 20) + 1), dict(K=0), dict(K=1025), dict(dtype=2), dict(tau=0.0),
                        dict(tau=-1.0), dict(tau=float("nan")), dict(tau=float("inf")), dict(tau=1e7)]),
}


def arguments(name):
    types, special, _, _ = CALLS[name]
    return {n: P if t is PTR else 8 for n, t in types} | {"dtype": 1, "out_dtype": 0, "bytes": 1 << 30, "stream": None} | special


@pytest.mark.parametrize("name", CALLS)
def test_refuses(lib, name):  # noqa: F811
    types, _, needed, bad = CALLS[name]
    for changed in bad + [{n: None} for n in needed.split()]:
        assert call(lib, name, types, arguments(name), **changed) == INVALID, changed


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("changed", [dict(ws=None), dict(ws=P + 128), dict(bytes=255)])
def test_workspace_refused(lib, name, changed):  # noqa: F811
    assert call(lib, name, CALLS[name][0], arguments(name), **changed) == WORKSPACE


@pytest.mark.parametrize("name,count", [("dspark_probabilities", "N"), ("dspark_page_copy", "n"), ("dspark_distill", "N")])
def test_nothing_to_do_is_no_error(lib, name, count):  # noqa: F811
    types = CALLS[name][0]
    nothing = {n: None if t is PTR and n != "ws" else arguments(name)[n] for n, t in types}
    assert call(lib, name, types, nothing, **{count: 0}) == 0


def test_page_workspace_size(lib):  # noqa: F811
    f = lib.dspark_page_workspace_bytes
    f.restype = SIZE
    assert f(0) == 0 and f(1) % 256 == 0 and f(1000) > f(10) > 0
    for name in ("dspark_page_collect", "dspark_page_fork", "dspark_page_compact"):
        assert call(lib, name, CALLS[name][0], arguments(name), bytes=f(8) - 1) == WORKSPACE


def test_binding_refuses_shapes():
    torch = pytest.importorskip("torch")
    from speculative_decoding_draft_seq_gb300 import dspark as d
    f, i, u8 = torch.zeros, lambda *s: torch.zeros(s, dtype=torch.int32), torch.zeros(256, dtype=torch.uint8)
    with pytest.raises(ValueError, match="temperature"):
        d.probabilities(f(3, 8), f(2), f(3, 8), u8)
    with pytest.raises(ValueError, match="probs"):
        d.probabilities(f(3, 8), f(3), f(3, 9), u8)
    with pytest.raises(ValueError, match="q_start"):
        d.verify_probs(f(5, 8), i(3), None, i(3, 2), f(3, 3), i(3, 3), i(3), f(3, 2), u8)
    with pytest.raises(ValueError, match="draft_probs"):
        d.verify_probs(f(5, 8), i(4), f(3, 2, 9), i(3, 2), f(3, 3), i(3, 3), i(3), f(3, 2), u8)
    with pytest.raises(ValueError, match="kv_len"):
        d.page_collect(i(3, 4), i(2), 16, i(9), i(9), i(1), u8)
    with pytest.raises(ValueError, match="parent"):
        d.page_fork(i(3, 4), i(3), i(1), None, 16, 9, i(2), i(2, 4), i(2), i(2), i(2), i(2), i(1), u8)
    with pytest.raises(ValueError, match="src"):
        d.page_compact(i(3, 4), i(3), 16, 9, i(3, 4), i(9), i(4), i(1), u8)
    with pytest.raises(ValueError, match="new_pinned"):
        d.page_compact(i(3, 4), i(3), 16, 9, i(3, 4), i(4), i(4), i(1), u8, pinned=i(2))
    with pytest.raises(ValueError, match="dst"):
        d.page_copy(i(2), i(3), f(4, 16, 1, 8), f(4, 16, 1, 8), u8)
    with pytest.raises(ValueError, match="teacher_lse"):
        d.distill(f(3, 8), i(3, 2), f(3, 2), 1.0, f(3), u8, teacher_lse=f(2))
    with pytest.raises(ValueError, match="grad"):
        d.distill(f(3, 8), i(3, 2), f(3, 2), 1.0, f(3), u8, grad=f(3, 9))
