"""Distillation with the teacher's normaliser where the drafter's unlisted entries lie far below the listed ones.

s_R, the unlisted entries' share, may then lie far below float32's range; ln s_R and the shares s_v / s_R do not. Bounds, with
`weight_error` the relative error of a weight over a float32 sum (test_gpu_target_pass): the loss has a logarithm's error for Z and
for the sum over the unlisted entries, 2^-24 of a distance (in nats) from the rate's rounding (2^-22 with the other
roundings of an exponent), and p_R = 1 - sum p, p within 2^-27 each, so 2^-26 of its factor ln p_R + 1 - ln s_R. Entries of the
gradient have their weights' and sums' errors, that of p_R, and half a step of their type."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import target_pass as O

pytestmark = pytest.mark.gpu

from test_gpu_target_pass import DTYPES, HALF_STEP, host, on, run_distill, weight_error  # noqa: E402

if torch.cuda.is_available():
    from speculative_decoding_draft_seq_gb300 import dspark

LN2 = math.log(2)


def check(x, ids, t, tau, lse, weight=None):
    """tau and all float32 inputs are taken as the values they are."""
    tau = float(np.float32(tau))
    loss, grad, status = run_distill(x, ids, t, tau, lse, weight)
    assert status == dspark.OK
    rows, dt = host(x), x.dtype
    for r in range(len(rows)):
        L, G, parts = O.distill(rows[r], ids[r], np.float32(t)[r], tau, np.float32(lse[r]))
        s, p, p_R, named, below = parts["s"], parts["p"], parts["p_rest"], parts["named"], parts["below"]
        w = 1.0 if weight is None else float(np.float32(weight[r]))
        out = ~named & np.isfinite(rows[r])
        y = -below[out]  # nats below the row's maximum
        M = y.max() if out.any() else 0.0
        part = np.exp(y - M)
        share_R = part / part.sum()
        mean_s, mean_p = (s * below).sum(), (p * np.where(p > 0, below, 0)).sum()
        e_z = weight_error(0.0, mean_s / LN2)
        # The sum over the unlisted entries is relative to the row's maximum, or to their own: the latter surely where it is below
        # 2^-66 of the row's, and the former's bounds are the wider ones. Weights below 2^-126 of either are 0.
        log2_z = (M + math.log(part.sum())) / LN2 if out.any() else 0.0
        own, least = ((M - y) / LN2, 1.0) if log2_z < -67 else (-y / LN2, 2.0 ** log2_z)
        e_rest = weight_error(0.0, (share_R * own).sum())
        e_left = 2.0 ** -26 * (1 + p.sum())
        bound = 2.0 ** -22 * (mean_p + mean_s + p_R * (share_R * -y).sum()) + e_z * (p.sum() + p_R) + p_R * e_rest + 2.0 ** -23 * abs(L) + 1e-30
        if p_R > 0:
            bound += e_left * (abs(math.log(p_R)) + 1 - M)
        if abs(L) < 3e38:
            assert abs(loss[r] - L) <= bound, (r, loss[r], L, bound)
        else:
            assert loss[r] == math.inf, (r, loss[r], L)
        e_s = weight_error(below / LN2, mean_s / LN2)
        bound = s * ((p.sum() + p_R) * e_s + e_left) + np.where(named, p * 2.0 ** -23, 0.0)
        bound[out] += share_R * (p_R * (weight_error(own, 0.0) + e_rest) + e_left)
        bound = bound * abs(w) / tau + HALF_STEP[dt] * np.abs(G * w) * (1 + 2.0 ** -8) + 2.0 ** -125 * (1 + abs(w) / tau * (1 + p_R / least))
        err = np.abs(grad[r] - G * w)
        assert (err <= bound * (1 + HALF_STEP[dt])).all(), (r, np.nanmax(err / bound), int(np.argmax(err - bound)))
    # the loss alone, and the gradient over the logits, are the same bits
    alone = run_distill(x, ids, t, tau, lse, back=False)
    over = run_distill(x.clone(), ids, t, tau, lse, weight, in_place=True)
    assert np.array_equal(alone[0], loss) and np.array_equal(over[0], loss) and np.array_equal(over[1], grad)
    return loss, grad


@pytest.mark.parametrize("dtype", DTYPES)
def test_small_worked_rows(dtype):
    """Entry 0 listed, the others 87 and more nats below it."""
    x = on(np.array([[0.0, -9.0, -9.5, -10.0]]), dtype)
    ids, t = np.array([[0]]), np.array([[0.0]])
    loss, grad = check(x, ids, t, 0.1, [-math.log(0.9)])
    # ln s_R = -90 + ln(1 + e^-5 + e^-10)
    assert abs(loss[0] - (0.9 * math.log(0.9) + 0.1 * (math.log(0.1) + 90 - math.log(1 + math.exp(-5) + math.exp(-10))))) < 1e-4
    assert np.allclose(grad[0], [1, -0.99326, -0.0066925, -4.5e-5], rtol=2.0 ** -7)
    x = on(np.array([[0.0, -0.87, -1.0]]), dtype)
    loss, grad = check(x, ids, t, 0.01, [-math.log(0.5)])
    assert np.allclose(grad[0, :2], [50, -50], rtol=2.0 ** -7) and -2e-4 < grad[0, 2] < -5e-5


# in nats below the largest listed entry: 2^-66 is 45.7, 2^-126 87.3
GAPS = [0.0, 5.0, 30.0, 41.0, 44.0, 45.7, 47.0, 50.0, 60.0, 80.0, 86.0, 87.0, 88.0, 90.0, 120.0, 800.0, 3000.0]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tau", [1e-6, 1e-4, 0.01, 0.1, 0.5, 1.0, 20.0])
# one CTA a row, many rows a cluster; several CTAs; eight; rows that are read twice; loose entries alone
@pytest.mark.parametrize("N,V,K", [(700, 400, 6), (3, 3001, 9), (17, 40003, 9), (2, 262151 + 9, 30), (34, 7, 3)])
def test_far_rests(dtype, tau, N, V, K):
    if V > 100000 and tau not in (1e-4, 1.0):
        pytest.skip("long rows at two temperatures")
    rng = np.random.default_rng(int(V + 1000 * tau))
    gap = np.array([GAPS[(r + (12 if N < 10 else 0)) % len(GAPS)] for r in range(N)])
    full = rng.normal(size=(N, V)) * 1.5 - gap[:, None]
    ids = np.stack([rng.permutation(V)[:K] for _ in range(N)])
    top = rng.normal(size=(N, K))
    np.put_along_axis(full, ids, top, 1)
    for r in range(0, N, 5):  # some entries masked, and listed ones as far below
        full[r, rng.integers(0, V, V // 3)] = -math.inf
        full[r, ids[r, 0]] = 1.0
        full[r, ids[r, 1:2]] = -gap[r]
    ids[3::7, -1] = ids[3::7, 0]  # an id that comes twice; a shorter list
    for r in range(5, N, 7):
        full[r, ids[r, -1]] = -gap[r]
        ids[r, -1] = -1
    x = on(full * tau, torch.float64).to(dtype)
    t = rng.normal(size=(N, K)) * tau
    share = rng.choice([0.1, 0.5, 0.9, 0.999], N)
    lse = np.log(np.exp(np.float32(t).astype(np.float64) / float(np.float32(tau))).sum(1) / share)
    weight = rng.choice([1.0, 1024.0, -0.5, 0.0], N)
    loss, grad = check(x, ids, t, tau, lse, weight)
    assert np.isfinite(grad).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shift", [1e4, -3e6, 1e9])
def test_far_rests_of_shifted_rows(dtype, shift):
    """Logits far from 0, where a weight's exponent is formed from the difference: one side of the row or both."""
    x = np.full((4, 600), -math.inf)
    x[0, :8] = shift
    x[0, 8:] = shift - 2.0 ** -6 * abs(shift)
    x[1, :8] = 0.0
    x[1, 8:] = -abs(shift)
    x[2, :8] = abs(shift)
    x[2, 8:] = 1.0
    x[3, :8] = shift
    x[3, 8:300] = -abs(shift) * 4
    x[3, 300:] = -abs(shift) * 4.03125
    ids = np.tile(np.arange(0, 8, 2), (4, 1))
    ids[2] = [0, 1, 2, 3]
    x[2, 4:8] = 0.5
    x[0, 1::2], x[1, 1:8:2], x[3, 1:8:2] = x[0, 100], x[1, 100], x[3, 100]
    t = np.tile([0.0, 0.5, -0.5, 1.0], (4, 1))
    check(on(x, torch.float64).to(dtype), ids, t, 1.0, np.log(np.exp(t).sum(1) / 0.7))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [600, 40000])
@pytest.mark.parametrize("tau", [0.5, 1.0, 4.0])
def test_a_rest_of_masked_entries(dtype, V, tau):
    """The whole rest at the type's lowest value: its distance times its share. At -inf: s_R is 0, and the rest counts for nothing."""
    low = float(torch.finfo(dtype).min)
    x = torch.full((3, V), low, dtype=dtype, device="cuda")
    x[:, 5:8] = torch.tensor([1.0, 2.0, -1.0], dtype=dtype, device="cuda")
    x[1, 300:500] = -math.inf
    x[2] = torch.where(x[2] == low, -math.inf, x[2].double()).to(dtype)
    ids, t = np.tile([5, 6, 7], (3, 1)), np.tile([1.0, 2.0, 0.0], (3, 1))
    lse = np.log(np.exp(t / tau).sum(1) / np.array([0.875, 0.75, 0.5]))
    loss, grad, status = run_distill(x, ids, t, tau, lse)
    assert status == dspark.OK
    for r in range(3):
        L, G, parts = O.distill(host(x)[r], ids[r], np.float32(t[r]), tau, np.float32(lse[r]))
        assert (parts["p_rest"] > 0) == (r < 2)
        if r < 2:
            # p_R > 0.1 within 2^-26 of 1, the distance's product with the rate within 2^-24: 2^-21 with the sum's roundings
            assert abs(loss[r] - L) <= 2.0 ** -21 * L and L > 1e37, (r, loss[r], L)
            out = host(x)[r] == low
            n = out.sum()
            assert np.abs(grad[r][out] + parts["p_rest"] / n / tau).max() <= (HALF_STEP[dtype] + 2.0 ** -19) / n / tau
        else:
            assert abs(loss[r] - L) <= 2.0 ** -18 * (1 + abs(L))
        assert np.abs(grad[r] - G).max() <= (HALF_STEP[dtype] + 2.0 ** -19) * (np.abs(G).max() + 2.0 ** -3)
    alone = run_distill(x, ids, t, tau, lse, back=False)
    assert np.array_equal(alone[0], loss)


def test_far_rests_replayed():
    """A captured call, replayed on other rows, some far and some not: the eager call's bits."""
    V, N, K = 9001, 40, 5
    rng = np.random.default_rng(0)
    xs, wants = [], []
    ids = np.stack([rng.permutation(V)[:K] for _ in range(N)])
    t = rng.normal(size=(N, K))
    lse = np.log(np.exp(t).sum(1) / 0.6)
    for far in ([0, 1, 17, 39], [2, 3, 4, 20]):
        full = rng.normal(size=(N, V))
        full[far] -= 100.0
        np.put_along_axis(full, ids, rng.normal(size=(N, K)), 1)
        xs.append(on(full, torch.float32))
        wants.append(check(xs[-1], ids, t, 1.0, lse))
    x, loss, grad = xs[0].clone(), torch.empty(N, device="cuda"), torch.empty_like(xs[0])
    ws = dspark.new_workspace(1, 1, 1, 1, dspark.FP32, 1)
    args = [on(ids, torch.int32), on(t, torch.float32)]
    teacher_lse = on(lse, torch.float32)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dspark.distill(x, *args, 1.0, loss, ws, grad=grad, teacher_lse=teacher_lse)
    for i in (0, 1, 1, 0):
        x.copy_(xs[i])
        g.replay()
        assert np.array_equal(host(loss), wants[i][0]) and np.array_equal(host(grad), wants[i][1])
    assert dspark.device_status(ws) == dspark.OK
