"""GPU tests of shared-prefix attention where it could go wrong: a wait that runs out, a token that takes
nearly all the weight, zero values beside small ones, large later tokens of a chunk, values that are not finite.
Helpers and the definition are those of test_gpu_prefix and prefix_testlib."""
import numpy as np
import pytest
import torch

from calibration_free_vector_b200 import nsn
import cache_testlib as ct
import prefix_testlib as pt
from test_gpu_prefix import SCALE, books, decode, extend, make, own_counts, queries, workspace

pytestmark = pytest.mark.gpu


def attend(q, k, v):
    """One softmax over the rows k / v [n, 128] for queries q [m, 128], in fp64 (numpy): (out, tolerance).

    Tolerance, where few tokens have the weight (prefix_testlib's terms, with hard bounds in place of multiples of
    a root mean square where one rounding counts alone; rho = 2^-11 / sqrt(3)):
      - weights: sum p_t |v_t - out| 6 ds_t with ds_t = 2 rho |q~ * y_t| + rho |s_t| + rho, as there, and 2^-32 of
        the largest weight for each token, where fp16 ends (half a step of 2^-24, weights scaled to 2^7 at least);
      - rows of V: 2^-11 of each for the scale that its dims share; two roundings per dim, the product with the mean
        (whose norm is below the row's in these tests) and the sum, which H spreads over the dims: six times
        sqrt(2) rho sqrt(sum p^2 |v_t|^2 / 128);
      - fp32 sums and the approximate exponential: 2^-22 of the largest element."""
    s = q @ k.T * SCALE
    p = np.exp(s - s.max(1, keepdims=True))
    top = 1.0 / p.sum(1, keepdims=True)
    p *= top
    out = p @ v
    h = pt.hadamard()
    ds = 2 * pt.RHO * np.sqrt(((q @ h * SCALE) ** 2) @ ((k @ h) ** 2).T) + pt.RHO * np.abs(s) + pt.RHO
    tol = np.stack([6 * (pi * di) @ np.abs(v - oi) for pi, di, oi in zip(p, ds, out)])
    tol += 2.0 ** -32 * top * np.abs(v).sum(0) + 2.0 ** -11 * p @ np.abs(v)
    tol += 6 * np.sqrt(2.0) * pt.RHO * np.sqrt((p ** 2) @ (v ** 2).sum(1, keepdims=True) / 128)
    return out, tol + np.abs(out).max(1, keepdims=True) * 2.0 ** -22


@pytest.mark.parametrize("B,g,dt,cap", [(4, 4, torch.bfloat16, None), (70, 8, torch.float16, None),
                                        (64, 4, torch.float32, 2304)])     # (the last: own parts by the decode kernel)
def test_a_wait_that_runs_out_gives_nan_and_a_status_bit(B, g, dt, cap):
    # one CTA gives up; the table entries and partials that it would have written are never read
    H = 2
    caches = make([(2560, 100), (1280, 0)], own_counts(B, H), 2, 1, False, seed=101, cap=cap)
    _, _, dk, dv = books(2, 1)
    q = queries((B, H * g, 128), dt, 22)
    want = decode(caches, q, dk, dv)
    ws = workspace(caches[0], caches[2], H * g)
    status = caches[2].status
    for cta in (0, 3, 1):
        out = torch.zeros_like(q)
        nsn.nsn_selftest_prefix_give_up(*caches, q, SCALE, dk, dv, out, ws, cta=cta)
        torch.cuda.synchronize()
        assert int(status.item()) == 2
        assert torch.isnan(out).all()
        status.zero_()
        nsn.nsn_decode_attention_prefix(*caches, q, SCALE, dk, dv, out, ws)     # the same workspace serves the next call
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        assert torch.equal(out, want)
    out = torch.zeros_like(q)
    nsn.nsn_selftest_prefix_give_up(*caches, q, SCALE, dk, dv, out, ws, cta=10**6)     # no such CTA: an ordinary call
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and torch.equal(out, want)


def test_give_up_refuses_a_negative_cta():
    caches = make([(128, 3)], [[(128, 3)]], 2, 2, False, seed=89)
    _, _, dk, dv = books(2, 2)
    q = queries((1, 4, 128), torch.bfloat16, 1)
    with pytest.raises(nsn.NsnError):
        nsn.nsn_selftest_prefix_give_up(*caches, q, SCALE, dk, dv, torch.empty_like(q),
                                        workspace(caches[0], caches[2], 4), cta=-1)


def test_a_first_token_that_takes_nearly_all_the_weight():
    # its key scores about 17.7 nats above the other 32767, its value is a twentieth of theirs, and theirs point the
    # same way.  256 query rows and 64 kv-heads: a partial runs over some 14k tokens.
    B, H, n, g = 256, 64, 32768, 1
    caches = make([(n, 0)] * H, [[(0, 0)] * H] * B, 2, 2, False, seed=111, s1_range=(0.2, 0.21), poison=False)
    pk, pv = caches[:2]
    pk.norms[:, :, 0, 0] = 1.0
    pv.norms[..., 0] = 1.0
    pv.norms[:, :, 0, 0] = 0.05
    pv.means[:] = pv.means[:, :, :1].clone() * 4
    cbk, cbv, dk, dv = books(2, 2)
    k0 = torch.empty((1, 1, H, 128), device="cuda")
    nsn.nsn_dequantize_kv(pk, k0, dk)
    lift = torch.linspace(17.5, 17.9, B, device="cuda")[:, None, None]
    q = k0[0, 0] / (k0[0, 0] ** 2).sum(-1, keepdim=True) * lift / SCALE
    out = decode(caches, q, dk, dv)
    for h in (0, 31, 63):
        want, tol = attend(q[:, h].double().cpu().numpy(), ct.rows(pk, 0, h, cbk, 2), ct.rows(pv, 0, h, cbv, 2))
        off = np.abs(out[:, h].double().cpu().numpy() - want) / tol
        assert off.max() <= 1, f"head {h}: {off.max():.3g} tolerances off"


@pytest.mark.parametrize("where", ["window", "block"])
def test_zero_values_beside_small_ones(where):
    # a token of value zero scores 12 nats above the others, whose values have norms of 1e-5 to 1e-4: it takes part
    # in the denominator only.  640 kv-heads: most items are whole in one CTA.
    B, H, g = 3, 640, 2
    caches = make([(384, 3)] * H, [[(0, 0)] * H] * B, 2, 2, False, seed=121)
    pk, pv = caches[:2]
    small = torch.rand(pv.norms.shape[:3], generator=torch.Generator().manual_seed(1)) * 9e-5 + 1e-5
    pv.norms[..., 0] = small.half().cuda()
    pv.window_buf.zero_()
    pv.norms[:, :, :128, 0] = 0
    cbk, cbv, dk, dv = books(2, 2)
    k = torch.empty((1, 387, H, 128), device="cuda")
    nsn.nsn_dequantize_kv(pk, k, dk)
    k0 = k[0, 385 if where == "window" else 5, :, None]
    lift = torch.linspace(11.5, 12.5, B * g, device="cuda").view(B, 1, g, 1)
    q = (k0 / (k0 ** 2).sum(-1, keepdim=True) * lift / SCALE).reshape(B, H * g, 128)
    out = decode(caches, q, dk, dv)
    for h in (0, 100, 333, 517, 639):
        qh, oh = (x[:, h * g:(h + 1) * g].reshape(B * g, 128).double().cpu().numpy() for x in (q, out))
        want, tol = attend(qh, ct.rows(pk, 0, h, cbk, 2), ct.rows(pv, 0, h, cbv, 2))
        off = np.abs(oh - want) / tol
        assert off.max() <= 1, f"head {h}: {off.max():.3g} tolerances off"


@pytest.mark.parametrize("B,C,g,own", [(2, 16, 4, [(128, 50), (0, 16)]), (1, 40, 8, [(256, 90)]), (3, 7, 1, [(0, 7), (128, 128), (0, 9)])])
def test_later_tokens_of_a_chunk_leave_earlier_queries_bit_for_bit(B, C, g, own):
    # finite rows up to 1500 times the others, infinities and NaN in the last tokens of the chunk: the queries before
    # them give the same bits (2048 is the documented limit)
    caches = make([(256, 40)], [[n] for n in own], 2, 2, False, seed=131)
    _, _, kc, vc = caches
    _, _, dk, dv = books(2, 2)
    q = queries((B, C, g, 128), torch.bfloat16, seed=23)
    clean = extend(caches, q, dk, dv)
    noise = torch.randn((2, 128), generator=torch.Generator().manual_seed(24)).cuda()
    for hidden in (1, C // 2):
        for size in (2e-4, 300.0, 1500.0, float("inf"), float("nan")):
            saved = [t.window_buf.clone() for t in (kc, vc)]
            for b, (_, nw) in enumerate(own):
                kc.window_buf[b, 0, nw - hidden:nw] = (noise[0] * size).half()
                vc.window_buf[b, 0, nw - hidden:nw] = (noise[1] * size).half()
            out = extend(caches, q, dk, dv)
            assert torch.equal(out[:, :C - hidden], clean[:, :C - hidden]), (hidden, size)
            kc.window_buf.copy_(saved[0])
            vc.window_buf.copy_(saved[1])


def test_a_later_value_400000_times_larger():
    # past the range in which not a bit changes: keys and values of root mean square 0.05, and a last token (K and V)
    # of 20000.  Its scale leaves the others 2^-9 of it: an element is off by 2^-25 / 2^-9 = 2^-16 of their root mean
    # square.  Keys: the score by at most six times |H q scale log2 e| 2^-16 / sqrt(3) 0.05 < 1e-5, and with it the
    # weights.  Values: 2^-16 each, which H spreads: 6 x 2^-16 / sqrt(3) of a root mean square at most.  Weights: the
    # reference is 9 (log2) higher, so a weight may differ by the half step 2^-25 where the largest is 2^-2: 2^-23 of
    # each value.  Normal weights and rows round alike (the scales are powers of two).
    C, g = 12, 4
    caches = make([(128, 0)], [[(128, 60)], [(0, 12)]], 2, 2, False, seed=141)
    _, pv, kc, vc = caches
    for c in (pv, vc):
        c.norms[..., 0] = 0.05
    for c in (kc, vc):
        c.window_buf.mul_(0.05)
    cbk, cbv, dk, dv = books(2, 2)
    q = queries((2, C, g, 128), torch.float32, seed=25)
    clean = extend(caches, q, dk, dv)
    for b, nw in enumerate((60, 12)):
        row = (torch.randn(128, generator=torch.Generator().manual_seed(b)) * 20000).clamp(-60000, 60000).half().cuda()
        vc.window_buf[b, 0, nw - 1] = kc.window_buf[b, 0, nw - 1] = row
    out = extend(caches, q, dk, dv)
    for b, nw in enumerate((60, 12)):
        v = np.concatenate([ct.rows(pv, 0, 0, cbv, 2), ct.rows(vc, b, 0, cbv, 2)[:-1]])
        tol = 1e-5 * np.abs(v).max() + 6 * 2.0 ** -16 / np.sqrt(3.0) * 0.05 + 2.0 ** -23 * np.abs(v).sum(0)
        off = np.abs((out[b, :C - 1] - clean[b, :C - 1]).cpu().numpy()) / tol
        assert off.max() <= 1, f"sequence {b}: {off.max():.3g} tolerances off"


INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("cap", [384, 2304])     # own parts as tiles, and by the decode kernel
@pytest.mark.parametrize("g,dt", [(1, torch.float32), (2, torch.float16), (4, torch.float32), (8, torch.bfloat16)])
def test_a_value_that_is_not_finite_gives_nan_whatever_the_capacity(g, dt, cap):
    # in own windows and own quantized tokens, keys and values: every query that sees one is NaN in all 128 dims, every
    # other one keeps its bits
    B, H = 64, 2
    own = [[(128 * ((b + h) % 3), 3 + (5 * b + h) % 120) for h in range(H)] for b in range(B)]
    caches = make([(256, 50), (128, 0)], own, 2, 1, False, seed=151, cap=cap)
    _, _, kc, vc = caches
    cbk, cbv, dk, dv = books(2, 1)
    q = queries((B, H * g, 128), dt, 26)
    clean = decode(caches, q, dk, dv)
    pt.check(*caches, q, clean, cbk, cbv, 2, 1, SCALE, pick={(b, h) for b in (0, 1, 2, 31, 63) for h in range(H)})
    # a key's infinity in the dim where the first query is largest, with the sign that makes its score minus infinity
    hot = q.view(B, H, g, 128)[:, :, 0].abs().argmax(-1)
    sign = -torch.sign(q.view(B, H, g, 128)[:, :, 0].float().gather(-1, hot[..., None]))[..., 0]
    bad = {}
    for i, (t, value) in enumerate([(kc, INF), (kc, NAN), (vc, INF), (vc, -INF), (vc, NAN)]):
        for j, row in enumerate((0, 2)):      # window rows
            b, h = 3 * i + j, (i + j) % H
            dim = int(hot[b, h])
            t.window_buf[b, h, row, dim] = value * float(sign[b, h]) if t is kc else value
            bad[b, h] = True
    for i, (t, name, value) in enumerate([(kc, "s1", INF), (kc, "s2", INF), (kc, "o", INF), (kc, "o", -INF), (kc, "s1", NAN),
                                          (vc, "s1", INF), (vc, "s2", INF), (vc, "o", INF), (vc, "s2", NAN)]):
        b, h = [(b, h) for b in range(20, B) for h in range(H) if own[b][h][0] and (b, h) not in bad][5 * i]
        if name == "o":
            t.means[b, h, 0, 77] = value
        else:
            t.norms[b, h, 100, 0 if name == "s1" else 1] = value
        bad[b, h] = True
    out = decode(caches, q, dk, dv)
    for b in range(B):
        for h in range(H):
            got, want = out[b, h * g:(h + 1) * g], clean[b, h * g:(h + 1) * g]
            if (b, h) in bad:
                assert torch.isnan(got).all(), (b, h)
            else:
                assert torch.equal(got, want), (b, h)


@pytest.mark.parametrize("which", ["key", "value"])
@pytest.mark.parametrize("dq", [False, True])
def test_a_block_whose_only_norms_are_nan(which, dq):
    # one token, or a block with zero norms beside it: nothing else sets the block's scale
    caches = make([(1, 0)], [[(1, 0)], [(128, 0)]], 2, 2, dq, seed=161, prefix_window=0, own_window=0)
    c = caches[2 if which == "key" else 3]
    _, _, dk, dv = books(2, 2)
    q = queries((2, 4, 128), torch.float32, 27)
    assert torch.isfinite(decode(caches, q, dk, dv)).all()
    if dq:
        c.dq_params[:, :, :, :2] = NAN
    else:
        c.norms[..., 0] = 0
        c.norms[:, :, 0, 0] = NAN
    assert torch.isnan(decode(caches, q, dk, dv)).all()


def test_an_infinity_through_the_quantizer():
    # as it would get there: a prompt with one infinite key (prefix), another with one infinite value (own cache)
    B, H, g, T = 2, 2, 4, 300
    _, _, dk, dv = books(2, 2)
    x = torch.randn((4, B, T, H, 128), generator=torch.Generator().manual_seed(28)).cuda()
    x[0, 0, 5, 0, 3] = INF
    x[3, 1, 200, 1, 9] = -INF
    pk, pv = nsn.Cache(1, H, 384, 0, 2), nsn.Cache(1, H, 384, 0, 2)
    kc, vc = nsn.Cache(B, H, 384, 128, 2), nsn.Cache(B, H, 384, 128, 2)
    for c, rows, book in ((pk, x[0, :1], dk), (pv, x[1, :1], dv), (kc, x[2], dk), (vc, x[3], dv)):
        nsn.nsn_quantize_kv(c, rows, book)
    out = decode((pk, pv, kc, vc), queries((B, H * g, 128), torch.float32, 29), dk, dv)
    nan = torch.isnan(out).view(B, H, g * 128)
    assert nan.all(-1).tolist() == [[True, False], [True, True]] and nan.any(-1).tolist() == [[True, False], [True, True]]


def test_broadcast_queries_and_many_row_tiles():
    # one query row for the whole batch (stride 0), 4800 rows a kv-head; the own parts differ
    B, H, g = 600, 1, 8
    caches = make([(640, 77)], [[(128 * (b % 2), b % 129)] for b in range(B)], 1, 2, True, seed=171)
    cbk, cbv, dk, dv = books(1, 2)
    q = queries((1, H * g, 128), torch.float16, 30).expand(B, H * g, 128)
    out = decode(caches, q, dk, dv)
    assert torch.equal(out, decode(caches, q.contiguous(), dk, dv))
    pt.check(*caches, q, out, cbk, cbv, 1, 2, SCALE, pick={(b, 0) for b in (0, 1, 31, 32, 33, 299, 598, 599)})
