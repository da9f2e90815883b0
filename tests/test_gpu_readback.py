"""GPU parity of reading a cache back (nsn_dequantize_kv) against the oracle's dequantization.

Tolerance, per element: the transform adds 128 terms whose absolute values sum to A
(cache_testlib.terms).  Sixteen of them are added by the tensor core (exact products, each
of 16 additions off by at most 2^-23 of A), then three butterfly stages and four scalings
(2^-24 each): less than 40 x 2^-24 A.  The final rounding adds half a step of the output
type, eps/2 |x| (2^-25 in fp16's subnormals)."""
import numpy as np
import pytest
import torch

from calibration_free_vector_b200 import nsn
import cache_testlib as ct
import nsn_testlib as tl

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16, torch.float16]
SENTINEL = 7.0


def check(cache, out, start, cb, mode, n=None):
    """Every row of out [B, T, H, 128] against the definition; rows past a sequence's end untouched."""
    got = out.float().cpu().numpy().astype(np.float64)
    for b in range(cache.batch):
        for h in range(cache.n_kv_heads):
            want, a = ct.rows(cache, b, h, cb, mode)[start:], ct.terms(cache, b, h, cb, mode)[start:]
            m = min(len(want), got.shape[1])
            want, a = want[:m], a[:m]
            tol = 40 * 2.0 ** -24 * a[:, None] + np.abs(want) * torch.finfo(out.dtype).eps / 2 + 2.0 ** -25
            bad = np.abs(got[b, :m, h] - want) > tol
            assert not bad.any(), f"(b={b}, h={h}) token {start + int(np.argwhere(bad)[0][0])}: {int(bad.sum())} values off"
            assert np.all(got[b, m:, h] == SENTINEL), f"(b={b}, h={h}): a row past the end was written"


@pytest.mark.parametrize("dq", [False, True])
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("mode", [1, 2])
def test_readback_ragged_counts(mode, dtype, dq):
    # several blocks, one block, window only, nothing, a full window
    counts = [[(1152, 128), (128, 5)], [(0, 77), (0, 0)], [(896, 0), (256, 1)]]
    cache = ct.random_cache(counts, 1152, 128, mode, dq, seed=10 * mode + dq)
    cb = tl.codebook(mode)
    out = torch.full((3, 1300, 2, 128), SENTINEL, dtype=dtype, device="cuda")
    before = [t.clone() for t in (cache.codes, cache.norms, cache.means, cache.window_buf, cache.n_quant)]
    nsn.nsn_dequantize_kv(cache, out, torch.from_numpy(cb).cuda())
    check(cache, out, 0, cb, mode)
    for a, b in zip(before, (cache.codes, cache.norms, cache.means, cache.window_buf, cache.n_quant)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("start,n", [(0, 1), (1, 1), (127, 2), (130, 300), (511, 128), (640, 9), (700, 1), (5000, 4)])
@pytest.mark.parametrize("mode,dq", [(1, False), (2, True)])
def test_readback_ranges(start, n, mode, dq):
    cache = ct.random_cache([[(640, 60), (512, 128)]], 1024, 128, mode, dq, seed=start + n)
    cb = tl.codebook(mode)
    out = torch.full((1, n, 2, 128), SENTINEL, dtype=torch.float32, device="cuda")
    nsn.nsn_dequantize_kv(cache, out, torch.from_numpy(cb).cuda(), start=start)
    check(cache, out, start, cb, mode)


@pytest.mark.parametrize("n", [1, 15, 16, 17, 127, 129, 1000])
def test_readback_without_window_ends_inside_a_block(n):
    cache = ct.random_cache([[(n, 0)]], 1024, 0, 2, False, seed=n)
    cb = tl.codebook(2)
    out = torch.full((1, 1024, 1, 128), SENTINEL, dtype=torch.bfloat16, device="cuda")
    nsn.nsn_dequantize_kv(cache, out, torch.from_numpy(cb).cuda())
    check(cache, out, 0, cb, 2)


def test_readback_strides_and_neighbours():
    # head-major rows, and K rows interleaved with V rows: nothing between the rows is written
    cache = ct.random_cache([[(256, 3)] * 3] * 2, 256, 128, 2, False, seed=5)
    cb = tl.codebook(2)
    dcb = torch.from_numpy(cb).cuda()
    big = torch.full((2, 3, 259, 128), SENTINEL, dtype=torch.float16, device="cuda")
    nsn.nsn_dequantize_kv(cache, big.transpose(1, 2), dcb)
    check(cache, big.transpose(1, 2), 0, cb, 2)
    kv = torch.full((2, 259, 3, 2, 128), SENTINEL, dtype=torch.bfloat16, device="cuda")
    nsn.nsn_dequantize_kv(cache, kv[:, :, :, 1], dcb)
    check(cache, kv[:, :, :, 1], 0, cb, 2)
    assert torch.all(kv[:, :, :, 0] == SENTINEL)


def test_readback_many_units_and_scales():
    # more blocks than resident warps (whole-block units), large and tiny norms
    counts = [[(16384, 128), (16000 - 16000 % 128, 40)] for _ in range(16)]
    cache = ct.random_cache(counts, 16384, 128, 2, False, seed=3, s1_range=(1e-3, 200.0))
    cb = tl.codebook(2)
    out = torch.full((16, 16512, 2, 128), SENTINEL, dtype=torch.float32, device="cuda")
    nsn.nsn_dequantize_kv(cache, out, torch.from_numpy(cb).cuda())
    for b in (0, 7, 15):
        for h in range(2):
            want, a = ct.rows(cache, b, h, cb, 2), ct.terms(cache, b, h, cb, 2)
            got = out[b, :, h].cpu().numpy().astype(np.float64)
            tol = 40 * 2.0 ** -24 * a[:, None] + np.abs(want) * 2.0 ** -24 + 2.0 ** -25
            assert not (np.abs(got[:len(want)] - want) > tol).any()
            assert np.all(got[len(want):] == SENTINEL)


def test_readback_on_a_stream_and_in_a_graph():
    cache = ct.random_cache([[(384, 100)]], 384, 128, 2, False, seed=8)
    cb = tl.codebook(2)
    dcb = torch.from_numpy(cb).cuda()
    out = torch.full((1, 484, 1, 128), SENTINEL, dtype=torch.float32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    nsn.nsn_dequantize_kv(cache, out, dcb, stream=side)
    side.synchronize()
    check(cache, out, 0, cb, 2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nsn.nsn_dequantize_kv(cache, out, dcb)
    out.fill_(SENTINEL)
    cache.n_quant.fill_(256)     # a replay reads the counters of its own time
    graph.replay()
    torch.cuda.synchronize()
    check(cache, out, 0, cb, 2)


def test_readback_of_what_the_quantizer_wrote():
    # prefill, appends across a flush, then read back: each token within the quantizer's own error, the window exact
    B, T, H = 2, 500, 2
    x = torch.randn((B, T + 40, H, 128), generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    cb = tl.codebook(2)
    dcb = torch.from_numpy(cb).cuda()
    kc, vc = nsn.Cache(B, H, 640, 128, 2), nsn.Cache(B, H, 640, 128, 2)
    nsn.nsn_quantize_kv(kc, x[:, :T], dcb)
    nsn.nsn_quantize_kv(vc, x[:, :T], dcb)
    for t in range(T, T + 40):
        nsn.nsn_append_residual(kc, vc, x[:, t], x[:, t], dcb, dcb)
    out = torch.full((B, T + 40, H, 128), SENTINEL, dtype=torch.float32, device="cuda")
    nsn.nsn_dequantize_kv(kc, out, dcb)
    check(kc, out, 0, cb, 2)
    nq = int(kc.n_quant[0, 0])
    assert torch.equal(out[:, nq:], x[:, nq:].half().float())     # the window holds fp16
    cos = torch.nn.functional.cosine_similarity(out[:, :nq], x[:, :nq].float(), dim=-1)
    assert float(cos.min()) > 0.8


def test_readback_past_32_bit_offsets():
    # records more than 4 GB into the buffers: the last tokens of the last of three long sequences
    cap, n = 1 << 27, 300
    cache = nsn.Cache(1, 3, cap, 0, 1)
    small = ct.random_cache([[(n, 0)]], 384, 0, 1, False, seed=77, poison=False)
    off = cap - 384
    cache.codes[0, 2, off:] = small.codes[0, 0]
    cache.norms[0, 2, off:] = small.norms[0, 0]
    cache.means[0, 2, off // 128:] = small.means[0, 0]
    cache.n_quant[0, 2] = off + n
    cb = tl.codebook(1)
    out = torch.full((1, 384, 3, 128), SENTINEL, dtype=torch.float32, device="cuda")
    nsn.nsn_dequantize_kv(cache, out, torch.from_numpy(cb).cuda(), start=off)
    check(small, out[:, :, 2:], 0, cb, 1)
    assert torch.all(out[:, :, :2] == SENTINEL)


def test_readback_refuses_what_it_cannot_take():
    cache = ct.random_cache([[(128, 3)]], 128, 128, 2, False, seed=1)
    dcb = torch.from_numpy(tl.codebook(2)).cuda()
    out = torch.empty((1, 131, 1, 128), dtype=torch.float32, device="cuda")
    call = nsn.nsn_dequantize_kv
    for bad in (dict(out=out[0]), dict(out=out[..., :64]), dict(out=torch.empty((2, 131, 1, 128), device="cuda")),
                dict(out=out.cpu()), dict(codebook=dcb.cpu()), dict(codebook=dcb.half()), dict(codebook=dcb[:100]),
                dict(start=-1), dict(start=2**32), dict(out=out.transpose(1, 3))):
        a = dict(out=out, codebook=dcb, start=0) | bad
        with pytest.raises(ValueError):
            call(cache, a["out"], a["codebook"], start=a["start"])
    with pytest.raises(TypeError):
        call(cache, out.double(), dcb)
    with pytest.raises(nsn.NsnError):
        call(cache, out[:, :1].expand(1, 131, 1, 128), dcb)     # every token onto one row
