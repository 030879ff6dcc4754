"""Page calls refuse outputs that share memory with their inputs or with each other (no GPU needed: those calls are refused
on the host), and take arrays that touch."""
import pytest

from test_serving_args import INVALID, P, PTR, call, lib  # noqa: F401
from test_target_pass_args import CALLS, arguments

STEP = 1 << 16
INPUTS = {"dspark_page_collect": "table kv_len pinned", "dspark_page_fork": "table kv_len parent fork_len free pinned",
          "dspark_page_compact": "table kv_len pinned"}
OUTPUTS = {"dspark_page_collect": "refs free n_free", "dspark_page_fork": "new_table new_len src dst tokens used",
           "dspark_page_compact": "new_table new_pinned src dst n_live"}
# entries of each, all counts being 8
SIZES = {"table": 64, "new_table": 64, "used": 1, "n_free": 1, "n_live": 1, "src": {"dspark_page_compact": 4}, "dst": {"dspark_page_compact": 4}}


def entries(name, what):
    n = SIZES.get(what, 8)
    return n.get(name, 8) if isinstance(n, dict) else n


def apart(name):
    """Arguments whose arrays lie far from each other (and are never followed)."""
    args = arguments(name)
    pointers = [n for n, t in CALLS[name][0] if t is PTR and n not in ("ws", "stream")]
    return args | {n: P + (i + 1) * STEP for i, n in enumerate(pointers)}


PAIRS = [(name, out, other) for name in OUTPUTS for out in OUTPUTS[name].split()
         for other in (INPUTS[name] + " " + OUTPUTS[name]).split() if other != out]


@pytest.mark.parametrize("name,out,other", PAIRS)
def test_refused(lib, name, out, other):  # noqa: F811
    args, types = apart(name), CALLS[name][0]
    there, mine, theirs = args[other], entries(name, out), entries(name, other)
    in_place = name == "dspark_page_compact" and (out, other) in (("new_table", "table"), ("new_pinned", "pinned"))
    # at its front (in place, where that is allowed: shifted by an entry), at its last entry, its first entry under the last of `out`
    for at in ([] if in_place else [there]) + [there + 4 * (theirs - 1)] * (theirs > 1) + [there - 4 * (mine - 1)] * (mine > 1):
        assert call(lib, name, types, args, **{out: at}) == INVALID, (out, other, at - there)


def test_lengths_in_place_are_refused(lib):  # noqa: F811
    args = apart("dspark_page_fork")
    assert call(lib, "dspark_page_fork", CALLS["dspark_page_fork"][0], args, new_len=args["kv_len"]) == INVALID


@pytest.mark.gpu
def test_arrays_side_by_side():
    """All arrays of a call next to each other in one buffer: taken, and the results of arrays far apart."""
    torch = pytest.importorskip("torch")
    from speculative_decoding_draft_seq_gb300 import dspark as d
    ws = d.new_page_workspace(9)

    def arrays(gap, *values):
        sizes = [len(v) if isinstance(v, list) else v for v in values]
        buffer = torch.full((sum(sizes) + gap * len(sizes),), -7, dtype=torch.int32, device="cuda")
        out, at = [], 0
        for v, n in zip(values, sizes):
            out.append(buffer[at:at + n])
            if isinstance(v, list):
                out[-1].copy_(torch.tensor(v, dtype=torch.int32))
            at += n + gap
        return out

    results = []
    for gap in (0, 64):
        table, kv_len, pinned, refs, free, n = arrays(gap, [4, 2, 7, 1], [6, 8], [3], 9, 9, 1)
        d.page_collect(table.view(2, 2), kv_len, 4, refs, free, n, ws, pinned=pinned)
        made = [refs.tolist(), free.tolist(), n.tolist()]
        table, kv_len, parent, free, new, *rest = arrays(gap, [4, 2, 7, 1], [6, 8], [0, 0, 1], [5, 6], 6, 3, 3, 3, 3, 1)
        d.page_fork(table.view(2, 2), kv_len, parent, None, 4, 9, free, new.view(3, 2), *rest, ws)
        made += [x.tolist() for x in (new, *rest)]
        table, kv_len, pinned, src, dst, n = arrays(gap, [4, 2, 7, 1], [6, 8], [8], 4, 4, 1)
        d.page_compact(table.view(2, 2), kv_len, 4, 9, table.view(2, 2), src, dst, n, ws, pinned=pinned, new_pinned=pinned)
        made += [x.tolist() for x in (table, kv_len, pinned, src, dst, n)]
        results.append(made)
    assert results[0] == results[1] and d.device_status(ws) == d.OK
