"""GPU parity of attention over a shared prefix and own caches (nsn_decode_attention_prefix,
nsn_extend_attention_prefix) against the definition in fp64; the tolerance is derived in
prefix_testlib."""
import math

import numpy as np
import pytest
import torch

from calibration_free_vector_b200 import nsn
import cache_testlib as ct
import nsn_testlib as tl
import prefix_testlib as pt

pytestmark = pytest.mark.gpu
SCALE = 1.0 / math.sqrt(128)
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def make(prefix, own, mk, mv, dq, seed, prefix_window=128, own_window=128, cap_p=None, cap=None, **kw):
    """(prefix K, prefix V, own K, own V): prefix [(nq, nw) per head], own [[(nq, nw) per head] per sequence]."""
    up = lambda counts: max(128, max(-(-n // 128) * 128 for row in counts for n, _ in row))  # noqa: E731
    a = lambda counts, cp, w, mode, s: ct.random_cache(counts, cp or up(counts), w, mode, dq, s, **kw)  # noqa: E731
    return (a([prefix], cap_p, prefix_window, mk, seed), a([prefix], cap_p, prefix_window, mv, seed + 1),
            a(own, cap, own_window, mk, seed + 2), a(own, cap, own_window, mv, seed + 3))


def books(mk, mv):
    return tl.codebook(mk), tl.codebook(mv), torch.from_numpy(tl.codebook(mk)).cuda(), torch.from_numpy(tl.codebook(mv)).cuda()


def queries(shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def workspace(pk, kc, n_q, chunk=1):
    ws = nsn.prefix_workspace(pk, kc, n_q, chunk)
    counters = -(-8 * kc.batch * kc.n_kv_heads // 256) * 256
    ws[counters:] = 255     # NaN past the counters: nothing may be read before it is written
    return ws


def decode(caches, q, dk, dv, out_dtype=None, scale=SCALE):
    out = torch.full(q.shape, float("nan"), dtype=out_dtype or q.dtype, device="cuda")
    nsn.nsn_decode_attention_prefix(*caches, q, scale, dk, dv, out, workspace(caches[0], caches[2], q.shape[1]))
    torch.cuda.synchronize()
    assert int(caches[2].status.item()) == 0
    return out


def extend(caches, q, dk, dv, out_dtype=None, status=0):
    out = torch.full(q.shape, float("nan"), dtype=out_dtype or q.dtype, device="cuda")
    nsn.nsn_extend_attention_prefix(*caches, q, SCALE, dk, dv, out, workspace(caches[0], caches[2], q.shape[2], q.shape[1]))
    torch.cuda.synchronize()
    assert int(caches[2].status.item()) == status
    return out


# ragged own counts, one pattern per (b, h): blocks and window, window only, nothing, one token
OWN = [(256, 128), (0, 77), (128, 0), (0, 0), (0, 1), (384, 5)]


def own_counts(B, H):
    return [[OWN[(b * H + h) % len(OWN)] for h in range(H)] for b in range(B)]


@pytest.mark.parametrize("B,H,g,mk,mv,dq,dt", [
    (1, 1, 1, 1, 1, False, "f32"),      # one row
    (4, 2, 4, 2, 2, False, "bf16"),     # 16 rows: the groups alternate tiles
    (3, 2, 8, 2, 1, True, "f16"),       # 24 rows, double quantization
    (33, 2, 4, 1, 2, False, "bf16"),    # 132 rows: a second, mostly empty, half
    (64, 1, 4, 2, 2, True, "bf16"),     # 256 rows
    (70, 1, 8, 1, 1, False, "f16"),     # 560 rows: two whole row tiles and a part
    (40, 2, 2, 2, 1, False, "f32"),
])
def test_decode_prefix(B, H, g, mk, mv, dq, dt):
    prefix = [(640, 128), (768, 3)][:H]
    caches = make(prefix, own_counts(B, H), mk, mv, dq, seed=B + g)
    cbk, cbv, dk, dv = books(mk, mv)
    q = queries((B, H * g, 128), DTYPES[dt], seed=B)
    out = decode(caches, q, dk, dv)
    pt.check(*caches, q, out, cbk, cbv, mk, mv, SCALE)


@pytest.mark.parametrize("prefix,window", [
    ([(0, 0), (0, 0)], 128), ([(0, 1), (0, 128)], 128), ([(128, 0), (0, 0)], 128), ([(1, 0), (1000, 0)], 0),
    ([(127, 0), (129, 0)], 0), ([(2560, 64), (128, 64)], 128)])
def test_decode_prefix_lengths(prefix, window):
    B, H, g, mk, mv = 5, 2, 4, 2, 2
    caches = make(prefix, own_counts(B, H), mk, mv, False, seed=7, prefix_window=window)
    cbk, cbv, dk, dv = books(mk, mv)
    q = queries((B, H * g, 128), torch.bfloat16, seed=3)
    out = decode(caches, q, dk, dv, torch.float32)
    for b in range(B):
        for h in range(H):
            if sum(prefix[h]) + sum(own_counts(B, H)[b][h]) == 0:
                assert torch.all(out[b, h * g:(h + 1) * g] == 0)     # no token at all: zeros
    pt.check(*caches, q, out, cbk, cbv, mk, mv, SCALE)


def test_decode_prefix_own_without_window():
    # own caches that quantize everything (window 0), ending inside a block
    own = [[(70, 0), (300, 0)], [(0, 0), (128, 0)]]
    caches = make([(512, 9), (384, 128)], own, 2, 1, True, seed=21, own_window=0)
    cbk, cbv, dk, dv = books(2, 1)
    q = queries((2, 8, 128), torch.float16, seed=4)
    pt.check(*caches, q, decode(caches, q, dk, dv), cbk, cbv, 2, 1, SCALE)


@pytest.mark.parametrize("own_window", [128, 0])
def test_decode_prefix_large_own_caches(own_window):
    # own caches whose capacity makes them the decode kernel's: long, short and empty ones
    B, H, g, mk, mv = 64, 2, 4, 2, 1
    own = [[(128 * ((5 * b + h) % 19), 0 if own_window == 0 else (31 * b + h) % 129) for h in range(H)] for b in range(B)]
    caches = make([(640, 50), (0, 0)], own, mk, mv, False, seed=37, cap=2304, own_window=own_window)
    cbk, cbv, dk, dv = books(mk, mv)
    q = queries((B, H * g, 128), torch.bfloat16, seed=14)
    ws = nsn.prefix_workspace(caches[0], caches[2], H * g)
    outs = []
    for _ in range(2):     # the counters are back at zero after a call
        out = torch.full(q.shape, float("nan"), dtype=torch.float32, device="cuda")
        nsn.nsn_decode_attention_prefix(*caches, q, SCALE, dk, dv, out, ws)
        outs.append(out)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1])
    pt.check(*caches, q, outs[0], cbk, cbv, mk, mv, SCALE, pick={(b, h) for b in range(0, B, 5) for h in range(H)})


def test_decode_prefix_many_pieces():
    # several tiles and items per CTA, row tiles that several CTAs share
    B, H, g, mk, mv = 48, 4, 8, 2, 2
    own = [[(128 * ((b + 3 * h) % 6), (17 * b) % 129) for h in range(H)] for b in range(B)]
    caches = make([(5120, 128), (4992, 0), (5120, 31), (256, 1)], own, mk, mv, False, seed=31)
    cbk, cbv, dk, dv = books(mk, mv)
    q = queries((B, H * g, 128), torch.bfloat16, seed=5)
    out = decode(caches, q, dk, dv)
    pt.check(*caches, q, out, cbk, cbv, mk, mv, SCALE, pick={(b, h) for b in (0, 1, 17, 31, 32, 47) for h in range(H)})
    assert torch.equal(out, decode(caches, q, dk, dv))     # the split of the work is fixed: the same bits again


@pytest.mark.parametrize("lo,hi,qs", [(1e-4, 1e-3, 1.0), (50.0, 400.0, 0.02), (0.01, 3.0, 4.0)])
def test_decode_prefix_scales(lo, hi, qs):
    # tiny and large norms, peaked scores: weights and rows keep their relative precision
    caches = make([(1280, 0)], [[(256, 0)], [(128, 0)]], 2, 2, False, seed=41, s1_range=(lo, hi))
    cbk, cbv, dk, dv = books(2, 2)
    q = queries((2, 4, 128), torch.float32, seed=6) * qs
    pt.check(*caches, q, decode(caches, q, dk, dv), cbk, cbv, 2, 2, SCALE)


def test_decode_prefix_zero_vectors():
    # blocks of zero vectors (s1 = 0), alone and next to others
    caches = make([(384, 20)], [[(128, 20)]], 2, 2, False, seed=43)
    for c in caches:
        c.norms[:, :, :128, 0] = 0
        if c.capacity > 200:
            c.norms[:, :, 200, 0] = 0
        c.window_buf.zero_()
    cbk, cbv, dk, dv = books(2, 2)
    q = queries((1, 4, 128), torch.bfloat16, seed=7)
    pt.check(*caches, q, decode(caches, q, dk, dv), cbk, cbv, 2, 2, SCALE)


@pytest.mark.parametrize("B,C,H,g,mk,mv,dq,dt", [
    (2, 1, 2, 4, 2, 2, False, "bf16"),
    (3, 5, 2, 2, 2, 1, True, "f16"),
    (2, 33, 1, 4, 1, 1, False, "bf16"),     # 132 own rows
    (2, 128, 2, 8, 2, 2, False, "bf16"),    # four own row tiles
    (1, 128, 1, 1, 1, 2, True, "f32"),
    (5, 9, 1, 8, 2, 2, False, "f16"),
])
def test_extend_prefix(B, C, H, g, mk, mv, dq, dt):
    own = [[(128 * ((b + h) % 3), min(128, C + 13 * ((b + 2 * h) % 4))) for h in range(H)] for b in range(B)]
    caches = make([(768, 100), (384, 128)][:H], own, mk, mv, dq, seed=B + C)
    cbk, cbv, dk, dv = books(mk, mv)
    q = queries((B, C, H * g, 128), DTYPES[dt], seed=C)
    out = extend(caches, q, dk, dv)
    pt.check(*caches, q, out, cbk, cbv, mk, mv, SCALE, chunk=C)


def test_extend_prefix_later_tokens_do_not_reach_earlier_queries():
    # infinities and NaN in the chunk's later tokens: earlier queries as if they were not there
    B, C, H, g = 2, 16, 1, 4
    caches = make([(256, 40)], [[(128, 50)], [(0, 16)]], 2, 2, False, seed=51)
    cbk, cbv, dk, dv = books(2, 2)
    q = queries((B, C, H * g, 128), torch.bfloat16, seed=8)
    clean = extend(caches, q, dk, dv)
    pt.check(*caches, q, clean, cbk, cbv, 2, 2, SCALE, chunk=C)
    pk, pv, kc, vc = caches
    kc.window_buf[0, 0, 50 - 6] = float("nan")        # token of query 10
    vc.window_buf[0, 0, 50 - 4, 7] = float("inf")     # token of query 12
    vc.window_buf[1, 0, 15] = float("nan")            # the last token of sequence 1
    out = extend(caches, q, dk, dv)
    finite = torch.isfinite(out).all(-1).all(-1)
    assert finite[0].tolist() == [True] * 10 + [False] * 6
    assert finite[1].tolist() == [True] * 15 + [False]
    ref = pt.check
    kc.window_buf[0, 0, 50 - 6], vc.window_buf[0, 0, 50 - 4], vc.window_buf[1, 0, 15] = 0.0, 0.0, 0.0
    got = out.clone()
    got[0, 10:], got[1, 15:] = 0, 0
    again = extend(caches, q, dk, dv)
    again[0, 10:], again[1, 15:] = 0, 0
    assert torch.allclose(got.float(), again.float(), rtol=0.02, atol=1e-3)
    full = extend(caches, q, dk, dv)
    ref(*caches, q, full, cbk, cbv, 2, 2, SCALE, chunk=C)


def test_extend_prefix_flags_a_window_shorter_than_the_chunk():
    # the first queries of the short sequence see the prefix and its quantized tokens only
    C, g = 8, 4
    caches = make([(256, 0)], [[(128, 20)], [(128, 5)], [(0, 0)]], 2, 2, False, seed=61)
    cbk, cbv, dk, dv = books(2, 2)
    q = queries((3, C, g, 128), torch.bfloat16, seed=9)
    out = extend(caches, q, dk, dv, status=8)
    pt.check(*caches, q, out, cbk, cbv, 2, 2, SCALE, chunk=C)


def test_prefix_agrees_with_the_whole_sequence_in_one_cache():
    # prefix + own tokens against nsn_decode_attention over one cache of both: a run as it is used,
    # from prompts through appends across a flush
    B, H, g, P, S = 3, 2, 4, 512, 200
    cbk, cbv, dk, dv = books(2, 2)
    gen = torch.Generator().manual_seed(15)
    x = torch.randn((2, 1, P, H, 128), generator=gen).bfloat16().cuda()
    y = torch.randn((2, B, S, H, 128), generator=gen).bfloat16().cuda()
    pk, pv = nsn.Cache(1, H, P, 0, 2), nsn.Cache(1, H, P, 0, 2)
    nsn.nsn_quantize_kv(pk, x[0], dk)
    nsn.nsn_quantize_kv(pv, x[1], dv)
    kc, vc = nsn.Cache(B, H, 256, 128, 2), nsn.Cache(B, H, 256, 128, 2)
    fk, fv = nsn.Cache(B, H, P + 256, 128, 2), nsn.Cache(B, H, P + 256, 128, 2)
    nsn.nsn_quantize_kv(kc, y[0, :, :100], dk)
    nsn.nsn_quantize_kv(vc, y[1, :, :100], dv)
    both = torch.cat([x.expand(2, B, P, H, 128), y], 2)
    nsn.nsn_quantize_kv(fk, both[0, :, :P + 100], dk)
    nsn.nsn_quantize_kv(fv, both[1, :, :P + 100], dv)
    for t in range(100, S):
        nsn.nsn_append_residual(kc, vc, y[0, :, t], y[1, :, t], dk, dv)
        nsn.nsn_append_residual(fk, fv, y[0, :, t], y[1, :, t], dk, dv)
    assert torch.equal(pk.codes[0], fk.codes[0, :, :P])     # the same blocks
    q = queries((B, H * g, 128), torch.bfloat16, seed=10)
    out = decode((pk, pv, kc, vc), q, dk, dv, torch.float32)
    want = torch.empty_like(out)
    nsn.nsn_decode_attention(fk, fv, q, SCALE, dk, dv, want, nsn.decode_workspace(fk, H * g))
    pt.check(pk, pv, kc, vc, q, out, cbk, cbv, 2, 2, SCALE)
    assert tl.attn_error(out.cpu().numpy(), want.cpu().numpy()) <= tl.ATTN_TOL
    C = 6
    qc = queries((B, C, H * g, 128), torch.bfloat16, seed=11)
    ext = extend((pk, pv, kc, vc), qc, dk, dv, torch.float32)
    pt.check(pk, pv, kc, vc, qc, ext, cbk, cbv, 2, 2, SCALE, chunk=C)
    wext = torch.empty_like(ext)
    nsn.nsn_extend_attention(fk, fv, qc, SCALE, dk, dv, wext, nsn.decode_workspace(fk, H * g))
    assert tl.attn_error(ext.cpu().numpy(), wext.cpu().numpy()) <= tl.ATTN_TOL


def test_prefix_strided_queries_streams_and_graphs():
    B, H, g = 6, 2, 4
    caches = make([(640, 128)] * H, own_counts(B, H), 2, 2, False, seed=71)
    cbk, cbv, dk, dv = books(2, 2)
    big = queries((B, 3, H * g, 256), torch.bfloat16, seed=12)
    q = big[:, 1, :, 128:]
    assert not q.is_contiguous()
    ws = workspace(caches[0], caches[2], H * g)
    out = torch.full((B, H * g, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    nsn.nsn_decode_attention_prefix(*caches, q, SCALE, dk, dv, out, ws, stream=side)
    side.synchronize()
    pt.check(*caches, q, out, cbk, cbv, 2, 2, SCALE)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nsn.nsn_decode_attention_prefix(*caches, q, SCALE, dk, dv, out, ws)
    for c in caches[2:]:
        c.n_quant.fill_(128)          # a replay reads the counters of its own time
        c.norms.fill_(1.0)
        c.means.fill_(0.25)
    out.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    pt.check(*caches, q, out, cbk, cbv, 2, 2, SCALE)


def test_prefix_without_any_token():
    caches = make([(0, 0)], [[(0, 0)], [(0, 0)]], 2, 2, False, seed=81)
    cbk, cbv, dk, dv = books(2, 2)
    assert torch.all(decode(caches, queries((2, 4, 128), torch.bfloat16, 1), dk, dv) == 0)
    assert torch.all(extend(caches, queries((2, 3, 4, 128), torch.bfloat16, 1), dk, dv, status=8) == 0)


def test_prefix_calls_on_two_streams():
    # two batches over one prefix at the same time, each with its own workspace
    B, H, g, C = 24, 2, 4, 40
    pk, pv, kc, vc = make([(5120, 100)] * H, own_counts(B, H), 2, 1, False, seed=83)
    own = [[(128 * (b % 2), 40 + 7 * h) for h in range(H)] for b in range(3)]
    _, _, kx, vx = make([(128, 0)] * H, own, 2, 1, False, seed=85)
    cbk, cbv, dk, dv = books(2, 1)
    q, qx = queries((B, H * g, 128), torch.bfloat16, 16), queries((3, C, H * g, 128), torch.float16, 17)
    want, wantx = decode((pk, pv, kc, vc), q, dk, dv), extend((pk, pv, kx, vx), qx, dk, dv)
    ws, wsx = workspace(pk, kc, H * g), workspace(pk, kx, H * g, C)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [(torch.empty_like(q), torch.empty_like(qx)) for _ in range(8)]
    torch.cuda.synchronize()
    for out, outx in outs:
        nsn.nsn_decode_attention_prefix(pk, pv, kc, vc, q, SCALE, dk, dv, out, ws, stream=streams[0])
        nsn.nsn_extend_attention_prefix(pk, pv, kx, vx, qx, SCALE, dk, dv, outx, wsx, stream=streams[1])
    torch.cuda.synchronize()
    for out, outx in outs:
        assert torch.equal(out, want) and torch.equal(outx, wantx)
    pt.check(pk, pv, kx, vx, qx, wantx, cbk, cbv, 2, 1, SCALE, chunk=C)


def test_extend_prefix_past_32_bit_offsets():
    # own caches whose later sequences start more than 4 GB into their buffers
    cap, C, g = 1 << 27, 2, 4
    small = make([(256, 0)] * 3, [[(256, 20), (128, 9), (384, 128)]], 1, 1, False, seed=87, poison=False)
    big = []
    for c in small[2:]:
        d = nsn.Cache(1, 3, cap, 128, 1)
        n = c.capacity
        d.codes[:, :, :n], d.norms[:, :, :n], d.means[:, :, :n // 128] = c.codes, c.norms, c.means
        d.window_buf.copy_(c.window_buf)
        d.n_quant.copy_(c.n_quant)
        d.n_window.copy_(c.n_window)
        big.append(d)
    cbk, cbv, dk, dv = books(1, 1)
    q = queries((1, C, 3 * g, 128), torch.bfloat16, 18)
    out = extend((*small[:2], *big), q, dk, dv)
    pt.check(*small, q, out, cbk, cbv, 1, 1, SCALE, chunk=C)


def test_prefix_refuses_what_it_cannot_take():
    caches = make([(128, 3)], [[(128, 3)], [(0, 9)]], 2, 2, False, seed=89)
    cbk, cbv, dk, dv = books(2, 2)
    q, out = queries((2, 4, 128), torch.bfloat16, 1), torch.empty((2, 4, 128), device="cuda")
    ws = workspace(caches[0], caches[2], 4)
    good = dict(q=q, out=out, ws=ws, dk=dk)
    for bad in (dict(q=q[:1], out=out[:1]), dict(q=q[0]), dict(q=q.cpu()), dict(out=out[:1]), dict(out=out.cpu()),
                dict(out=torch.empty((4, 2, 128), device="cuda").transpose(0, 1)), dict(dk=dk.cpu()), dict(dk=dk.half()),
                dict(q=q[..., :64]), dict(ws=ws[::2])):
        a = good | bad
        with pytest.raises(ValueError):
            nsn.nsn_decode_attention_prefix(*caches, a["q"], SCALE, a["dk"], dv, a["out"], a["ws"])
    for bad in (dict(ws=ws[:-256]), dict(ws=ws[16:])):
        a = good | bad
        with pytest.raises(nsn.NsnError):
            nsn.nsn_decode_attention_prefix(*caches, a["q"], SCALE, a["dk"], dv, a["out"], a["ws"])
    with pytest.raises(nsn.NsnError):     # the own caches' batch is not 1
        nsn.nsn_decode_attention_prefix(caches[2], caches[3], *caches[2:], q, SCALE, dk, dv, out, ws)
    with pytest.raises(ValueError):
        nsn.prefix_workspace(caches[0], caches[2], 6)


def test_one_workspace_serves_decode_and_chunks_in_turn():
    # own caches large enough for the decode kernel, whose counters stay at zero through the chunk calls
    B, H, g, C = 64, 2, 4, 12
    own = [[(128 * ((b + h) % 4), 12 + (b + 5 * h) % 100) for h in range(H)] for b in range(B)]
    caches = make([(384, 7), (256, 128)], own, 2, 2, False, seed=91, cap=2304)
    cbk, cbv, dk, dv = books(2, 2)
    size = max(nsn.nsn_prefix_workspace_bytes(caches[0], caches[2], H * g, n) for n in (1, C))
    ws = torch.zeros((size,), dtype=torch.uint8, device="cuda")
    q1, qc = queries((B, H * g, 128), torch.bfloat16, 19), queries((B, C, H * g, 128), torch.bfloat16, 20)
    got = []
    for _ in range(2):
        o1, oc, oe = torch.empty_like(q1), torch.empty_like(qc), torch.empty_like(q1)
        nsn.nsn_decode_attention_prefix(*caches, q1, SCALE, dk, dv, o1, ws)
        nsn.nsn_extend_attention_prefix(*caches, qc, SCALE, dk, dv, oc, ws)
        nsn.nsn_extend_attention_prefix(*caches, q1[:, None], SCALE, dk, dv, oe[:, None], ws)
        got.append((o1, oc, oe))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert torch.equal(got[0][0], got[0][2])     # a chunk of one is a decode step
    pick = {(b, h) for b in (0, 9, 33, 63) for h in range(H)}
    pt.check(*caches, q1, got[0][0], cbk, cbv, 2, 2, SCALE, pick=pick)
    pt.check(*caches, qc, got[0][1], cbk, cbv, 2, 2, SCALE, chunk=C, pick=pick)


def test_decode_prefix_in_a_graph_with_large_own_caches():
    # three overlapping launches behind the decode kernel, captured and replayed
    B, H, g = 64, 2, 4
    own = [[(128 * ((b + h) % 3), (b + 5 * h) % 100) for h in range(H)] for b in range(B)]
    caches = make([(640, 7)] * H, own, 2, 1, True, seed=93, cap=2304)
    cbk, cbv, dk, dv = books(2, 1)
    q = queries((B, H * g, 128), torch.float16, 21)
    ws = nsn.prefix_workspace(caches[0], caches[2], H * g)
    want, out = torch.empty_like(q), torch.empty_like(q)
    nsn.nsn_decode_attention_prefix(*caches, q, SCALE, dk, dv, want, ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(3):
            nsn.nsn_decode_attention_prefix(*caches, q, SCALE, dk, dv, out, ws)
    for _ in range(3):
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
