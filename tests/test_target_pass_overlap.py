"""Probabilities, verification and distillation refuse outputs that share memory with their inputs or with each other (no GPU
needed: every call here is refused on the host)."""
import pytest

from test_serving_args import INVALID, P, PTR, call, lib  # noqa: F811, F401
from test_target_pass_args import CALLS, arguments

STEP = 1 << 16
# bytes of each array: all counts are 8, logits, gradients and rows of probabilities bf16, dspark_probabilities' results float32
BYTES = {"dspark_probabilities": ({"logits": 128, "temperature": 32}, {"probs": 256}),
         "dspark_verify_probs": ({"target": 128, "q_start": 36, "draft": 1024, "tokens": 256, "u": 576},
                                 {"out": 288, "accepted": 32, "p_tok": 256}),
         "dspark_distill": ({"logits": 128, "ids": 256, "teacher": 256, "lse": 32, "weight": 32}, {"loss": 32, "grad": 128})}
PAIRS = [(name, out, other) for name, (inputs, outputs) in BYTES.items() for out in outputs for other in [*inputs, *outputs] if other != out]


@pytest.mark.parametrize("name,out,other", PAIRS)
def test_refused(lib, name, out, other):  # noqa: F811
    inputs, outputs = BYTES[name]
    sizes, types = inputs | outputs, CALLS[name][0]
    args = arguments(name) | {n: P + (i + 1) * STEP for i, n in enumerate(n for n, t in types if t is PTR and n in sizes)}
    there = args[other]
    in_place = (name, out, other) == ("dspark_distill", "grad", "logits")
    # its front (where in place is allowed: one entry further), its last 2 bytes, its first 2 under the last ones of `out`
    for at in [there + (2 if in_place else 0), there + sizes[other] - 2, there - sizes[out] + 2]:
        assert call(lib, name, types, args, **{out: at}) == INVALID, at - there


def test_results_over_logits_of_another_type_are_refused(lib):  # noqa: F811
    types = CALLS["dspark_probabilities"][0]
    for a, b in ((0, 1), (1, 0)):
        args = arguments("dspark_probabilities") | {"logits": P, "probs": P, "temperature": P + STEP}
        assert call(lib, "dspark_probabilities", types, args, dtype=a, out_dtype=b) == INVALID


def test_losses_over_the_logits_of_a_call_in_place_are_refused(lib):  # noqa: F811
    args = arguments("dspark_distill") | {n: P + i * STEP for i, n in enumerate("ids teacher lse weight".split())}
    args |= {"logits": P + 9 * STEP, "grad": P + 9 * STEP, "loss": P + 9 * STEP + 64}
    assert call(lib, "dspark_distill", CALLS["dspark_distill"][0], args) == INVALID
