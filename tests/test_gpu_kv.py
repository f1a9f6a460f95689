"""The quantised key-value cache on the GPU: codes and scales bit for bit against their definition, attention against
64 bits.

Attention tolerance.  Scores: the codes and the scaled q are exact in fp16 (fp32 q: two fp16 terms, 2^-22 of the row's
largest value), sums are fp32 over d products, so a score is off by at most
  ds = scale * (d + 2) * 2^-23 * sum |q k|  (fp32 q: + scale * d * 2^-22 max|q| max|k|),
the exponential by 2^-22 more; an error of ds in the scores moves the weighted mean by at most 2 (e^ds - 1) max|v|.
Weights are rounded to fp16: 2^-11 of themselves (fp32: two terms, 2^-22), or 2^-25 of the largest weight where
that is more, for each token.  fp32 sums over n tokens: n 2^-23.  The output is rounded once to its type.
"""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def stepq():
    from quantized_recurrent_state_b200 import build as qbuild
    qbuild.build()
    from quantized_recurrent_state_b200 import stepq as s
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return s


def _randn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def _quantise(x, bits):
    """(codes, scales) as the header defines them, in 64 bits up to the stated roundings."""
    qmax = 2 ** (bits - 1) - 1
    x = x.double()
    r = (x.abs().amax(-1) / torch.tensor(float(qmax), dtype=torch.float64, device="cuda")).float()
    r = torch.where(r < 2.0 ** -126, torch.ones_like(r), r)
    z = torch.round(x * (1.0 / r).double().unsqueeze(-1)).clamp(-qmax, qmax)
    ok = torch.isfinite(x).all(-1)
    return torch.where(ok.unsqueeze(-1), z, torch.zeros_like(z)), torch.where(ok, r, torch.full_like(r, float("nan")))


class Seqs:
    """Sequences of the given lengths on shuffled pages."""

    def __init__(self, stepq, lens, bits, H, d, page, seed=1, spare=2):
        self.lens_list, self.page, self.H, self.d, self.bits = lens, page, H, d, bits
        pages = [-(-max(n, 0) // page) for n in lens]
        self.n_pages = sum(pages) + spare
        self.max_pages = max(pages + [1])
        order = torch.randperm(self.n_pages, generator=torch.Generator().manual_seed(seed)).tolist()
        table = torch.full((len(lens), self.max_pages), 10 ** 6, dtype=torch.int32)     # what is not used is never read
        for i, c in enumerate(pages):
            for j in range(c):
                table[i, j] = order.pop()
        self.table = table.cuda()
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.cu_list = [0]
        for n in lens:
            self.cu_list.append(self.cu_list[-1] + max(n, 0))
        self.cu = torch.tensor(self.cu_list, dtype=torch.int32, device="cuda")
        self.places = torch.tensor([int(table[i, t // page]) * page + t % page for i, n in enumerate(lens) for t in range(n)],
                                   dtype=torch.int64, device="cuda")
        self.kv = stepq.KVCache(bits, H, d, page, self.n_pages)
        self.cache = torch.randint(0, 256, (self.kv.bytes,), dtype=torch.uint8, device="cuda",
                                   generator=torch.Generator(device="cuda").manual_seed(seed))   # any contents will do
        self.total = self.cu_list[-1]

    def fill(self, k, v):
        self.kv.append(self.cache, k, v, self.places)

    def read(self, dtype):
        k, v = (torch.full((self.total, self.H, self.d), 7.0, dtype=dtype, device="cuda") for _ in range(2))
        self.kv.read(self.cache, self.table, self.lens, self.cu, k, v)
        self.kv.check()
        return k, v


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
def test_written_and_read_back(stepq, bits, d, dtype):
    H, lens = 3, [1, 0, 16, 37, 130]
    s = Seqs(stepq, lens, bits, H, d, 32)
    wide = (_randn(2, s.total, 2 * H + 1, d) * torch.exp2(6 * _randn(3, s.total, 2 * H + 1, 1)).clamp(2 ** -9, 2 ** 9)).to(TYPES[dtype])
    wide[5, 0] = 0.0                                     # a row of zeros
    wide[6, 0] = 0.0
    wide[6, 0, 3] = torch.finfo(TYPES[dtype]).tiny       # one small value in a row of zeros
    wide[7, 0] = torch.arange(d, device="cuda").to(TYPES[dtype]) % 15 - 7   # ties of 4-bit codes
    wide[7, 0, 0] = 14.0
    k, v = wide[:, :H], wide[:, H + 1:]                  # slices of a wider row
    s.fill(k, v)
    for out in ("fp32", "fp16", "bf16"):
        for x, got in zip((k, v), s.read(TYPES[out])):
            z, r = _quantise(x, bits)
            assert torch.equal(got, (r.unsqueeze(-1) * z.float()).to(TYPES[out]))


@pytest.mark.parametrize("bits", [8, 4])
def test_codes_are_where_the_header_says(stepq, bits):
    H, d, page = 2, 64, 16
    s = Seqs(stepq, [20], bits, H, d, page)
    k, v = _randn(4, 20, H, d), _randn(5, 20, H, d)
    before = s.cache.clone()
    s.fill(k, v)
    s.kv.check()
    rb = d * bits // 8
    head = page * (2 * rb + 8)
    seen = torch.zeros(s.kv.bytes, dtype=torch.bool)
    raw, table = s.cache.cpu(), s.table.cpu()
    for which, x in enumerate((k, v)):
        z, r = (y.cpu() for y in _quantise(x, bits))
        for t in range(20):
            for h in range(H):
                base = int(table[0, t // page]) * head * H + h * head
                c0 = base + which * page * rb + (t % page) * rb
                row = raw[c0:c0 + rb].int()
                u = row if bits == 8 else torch.stack([row & 15, row >> 4], -1).flatten()
                assert torch.equal(u - (1 << (bits - 1)), z[t, h].int())
                s0 = base + page * 2 * rb + which * page * 4 + (t % page) * 4
                assert raw[s0:s0 + 4].view(torch.float32).item() == r[t, h].item()
                seen[c0:c0 + rb] = True
                seen[s0:s0 + 4] = True
    assert torch.equal(raw[~seen], before.cpu()[~seen])  # nothing else was written


def test_rows_that_are_not_finite(stepq):
    s = Seqs(stepq, [4], 8, 1, 64, 16)
    k = _randn(6, 4, 1, 64)
    k[1, 0, 5] = float("inf")
    k[2, 0, 63] = float("nan")
    s.fill(k, k)
    got, _ = s.read(torch.float32)
    assert torch.isnan(got[1]).all() and torch.isnan(got[2]).all() and torch.isfinite(got[[0, 3]]).all()


def test_places_padding_and_range(stepq):
    s = Seqs(stepq, [32], 8, 2, 64, 16)
    k = _randn(7, 32, 2, 64)
    s.fill(k, k)
    s.kv.check()
    before = s.cache.clone()
    places = s.places.clone()
    places[3:] = stepq.PAD
    s.kv.append(s.cache, k, k, places)
    s.kv.check()
    assert torch.equal(s.cache, before)                  # the same rows again, the rest skipped
    for bad in (-2, s.n_pages * s.page, 1 << 40):
        places[5] = bad
        s.kv.append(s.cache, k * 2, k * 2, torch.where(places >= 0, places, places).where(torch.arange(32, device="cuda") >= 3,
                                                                                         torch.full_like(places, -1)))
        with pytest.raises(stepq.StepqError, match="out of range"):
            s.kv.check()
        assert torch.equal(s.cache, before)
    s.kv.check()                                         # the word was cleared
    s.kv.append(s.cache, k[:0], k[:0], places[:0])


def _attend(s, q, scale=None, lse=True):
    n, n_tok, hq, d = q.shape
    o = torch.full_like(q, 7.0)
    l = torch.full((n, n_tok, hq), 7.0, device="cuda") if lse else None
    ws = torch.empty(s.kv.attend_workspace_bytes(n, n_tok, hq, s.max_pages), dtype=torch.uint8, device="cuda")
    s.kv.attend(s.cache, q, s.table, s.lens, d ** -0.5 if scale is None else scale, o, ws, lse=l)
    s.kv.check()
    return o, l


def _check_attend(s, q, o, l, k, v, scale):
    """o, l against 64 bits from the values that the cache holds; returns the largest error over its bound."""
    n, n_tok, hq, d = q.shape
    dt = str(q.dtype).replace("torch.", "")
    wt = 2.0 ** -22 if dt == "float32" else 2.0 ** -11
    kd, vd = (r.double().unsqueeze(-1) * z.double() for z, r in (_quantise(k, s.bits), _quantise(v, s.bits)))
    rv = _quantise(v, s.bits)[1].double()
    rep, worst = hq // s.H, 0.0
    for i, length in enumerate(s.lens_list):
        if length < 0:
            assert (o[i] == 7.0).all() and (l is None or (l[i] == 7.0).all())
            continue
        for t in range(n_tok):
            m = length - n_tok + 1 + t
            if m <= 0:
                assert (o[i, t] == 0).all() and (l is None or (l[i, t] == -math.inf).all())
                continue
            sl = slice(s.cu_list[i], s.cu_list[i] + m)
            kk, vv = (x[sl].repeat_interleave(rep, 1) for x in (kd, vd))
            r = rv[sl].repeat_interleave(rep, 1)
            qq = q[i, t].double()
            sc = torch.einsum("hd,mhd->hm", qq, kk) * scale
            ref_l = torch.logsumexp(sc, -1)
            p = torch.exp(sc - ref_l.unsqueeze(-1))
            ref = torch.einsum("hm,mhd->hd", p, vv)
            ds = scale * (d + 2) * 2.0 ** -23 * torch.einsum("hd,mhd->hm", qq.abs(), kk.abs()).amax(-1)
            if dt == "float32":
                ds = ds + scale * d * 2.0 ** -22 * qq.abs().amax(-1) * kk.abs().amax((0, 2))
            ds = ds + 2.0 ** -22 + 2.0 ** -23 * sc.abs().amax(-1)      # the exponent itself is an fp32 number
            vmax = vv.abs().amax((0, 2))
            mean = torch.einsum("hm,mhd->hd", p, vv.abs())
            tiny = m * 2.0 ** -25 * 127 * (p.transpose(0, 1) * r).amax(0)
            bound = (2 * torch.expm1(ds) * vmax + tiny).unsqueeze(-1) + (wt + m * 2.0 ** -23) * mean
            bound = bound + torch.finfo(q.dtype).eps / 2 * (ref.abs() + bound) + (2.0 ** -25 if dt == "float16" else 0.0)
            err = (o[i, t].double() - ref).abs()
            assert (err <= bound).all(), (i, t, (err / bound).max().item())
            worst = max(worst, (err / bound).max().item())
            if l is not None:
                lb = ds + m * 2.0 ** -23 + 2.0 ** -22 * ref_l.abs()
                assert ((l[i, t].double() - ref_l).abs() <= lb).all()
    return worst


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("hq, n_tok", [(2, 1), (6, 2), (14, 1), (16, 5)])
def test_attend(stepq, bits, d, dtype, hq, n_tok):
    lens = [1, 0, 2, 17, 64, 301, -1, 130]
    s = Seqs(stepq, lens, bits, 2, d, 16 if d == 64 else 48)
    k, v = _randn(8, s.total, 2, d), _randn(9, s.total, 2, d)
    s.fill(k, v)
    q = _randn(10, len(lens), n_tok, hq, d).to(TYPES[dtype])
    o, l = _attend(s, q)
    _check_attend(s, q, o, l, k, v, d ** -0.5)


@pytest.mark.parametrize("bits, d, page", [(8, 128, 64), (4, 128, 16), (8, 64, 128), (4, 256, 32)])
def test_attend_long_is_split_and_joined(stepq, bits, d, page):
    lens = [5000, 33, 0, 9001]
    s = Seqs(stepq, lens, bits, 1, d, page)
    k, v = _randn(11, s.total, 1, d), _randn(12, s.total, 1, d)
    k[4000] *= 30.0                                      # one token that outweighs what came before it
    s.fill(k, v)
    q = _randn(13, len(lens), 1, 4, d).bfloat16()
    o, l = _attend(s, q)
    _check_attend(s, q, o, l, k, v, d ** -0.5)
    again, l2 = _attend(s, q)
    assert torch.equal(o, again) and torch.equal(l, l2)  # the joining order is fixed


@pytest.mark.parametrize("bits, d, page", [(8, 256, 32), (4, 64, 16), (8, 128, 64)])
def test_attend_repeats_bit_for_bit_under_load(stepq, bits, d, page):
    """Many long sequences keep every copy stage busy: a stage given back before it is read shows as runs that differ."""
    lens = [20000, 11947, 6743, 12999, 2549, 16789, 11102, 7387]
    s = Seqs(stepq, lens, bits, 2, d, page)
    k, v = _randn(40, s.total, 2, d).bfloat16(), _randn(41, s.total, 2, d).bfloat16()
    s.fill(k, v)
    q = _randn(42, len(lens), 1, 16, d).bfloat16()
    o, l = _attend(s, q)
    for _ in range(40):
        again, l2 = _attend(s, q)
        assert torch.equal(o, again) and torch.equal(l, l2)
    _check_attend(s, q, o, l, k, v, d ** -0.5)


def test_attend_scales_of_all_sizes(stepq):
    """Value rows from 2^-40 to 2^40, keys whose scores differ by hundreds: weights in fp16 have to stand it."""
    lens = [400]
    s = Seqs(stepq, lens, 8, 1, 128, 16)
    k = _randn(14, 400, 1, 128) * 4
    v = _randn(15, 400, 1, 128) * torch.exp2(80 * torch.rand(400, 1, 1, device="cuda", generator=torch.Generator(
        device="cuda").manual_seed(16)) - 40)
    s.fill(k, v)
    for dtype in ("fp32", "bf16"):
        q = (_randn(17, 1, 1, 8, 128) * 8).to(TYPES[dtype])
        o, l = _attend(s, q)
        _check_attend(s, q, o, l, k, v, 128 ** -0.5)
    s.fill(k, _randn(18, 400, 1, 128) * 1e30)            # large values everywhere
    q = _randn(19, 1, 1, 8, 128)
    o, l = _attend(s, q)
    _check_attend(s, q, o, l, k, _randn(18, 400, 1, 128) * 1e30, 128 ** -0.5)


def test_attend_what_is_masked_does_not_matter(stepq):
    """NaN rows behind the length, and between a draft's tokens, reach only the tokens that see them."""
    s = Seqs(stepq, [70], 8, 1, 64, 32)
    k, v = _randn(20, 70, 1, 64), _randn(21, 70, 1, 64)
    s.fill(k, v)
    q = _randn(22, 1, 3, 4, 64).half()
    clean, lclean = _attend(s, q)
    bad = torch.full((1, 1, 64), float("nan"), device="cuda")
    for t in range(70, 96):                              # the rest of the last page
        s.kv.append(s.cache, bad, bad, torch.tensor([int(s.table[0, 2]) * 32 + t - 64], device="cuda"))
    o, l = _attend(s, q)
    assert torch.equal(o, clean) and torch.equal(l, lclean)
    s.kv.append(s.cache, bad, bad, s.places[69:70])      # the newest token: only the last query sees it
    o, l = _attend(s, q)
    assert torch.equal(o[:, :2], clean[:, :2]) and torch.isnan(o[:, 2]).all() and torch.isnan(l[:, 2]).all()


def test_attend_bad_lengths_and_pages(stepq):
    s = Seqs(stepq, [40, 20], 8, 2, 64, 16)
    k = _randn(23, 60, 2, 64)
    s.fill(k, k)
    q = _randn(24, 2, 1, 2, 64)
    good, _ = _attend(s, q)
    s.lens[1] = s.max_pages * 16 + 1
    with pytest.raises(stepq.StepqError, match="length above"):
        _attend(s, q)
    s.lens[1] = 20
    s.table[1, 1] = s.n_pages
    with pytest.raises(stepq.StepqError, match="out of range"):
        _attend(s, q)
    with pytest.raises(stepq.StepqError, match="out of range"):
        s.read(torch.float32)
    s.table[1, 1] = -7
    with pytest.raises(stepq.StepqError, match="out of range"):
        _attend(s, q)
    s.lens[1] = 16                                       # the bad page is no longer used
    o, _ = _attend(s, q)
    assert torch.equal(o[0], good[0])


def test_read_leaves_other_rows(stepq):
    s = Seqs(stepq, [20, -1, 5], 4, 1, 128, 16)
    k = _randn(25, 25, 1, 128)
    s.fill(k, k)
    whole = torch.full((48, 2, 128), 7.0, device="cuda")
    out = whole[:40]
    cu = torch.tensor([10, 0, 33], dtype=torch.int32, device="cuda")
    s.kv.read(s.cache, s.table, s.lens, cu, out[:, :1], out[:, 1:])
    s.kv.check()
    z, r = _quantise(k, 4)
    x = r.unsqueeze(-1) * z.float()
    assert torch.equal(out[10:30, :1], x[:20]) and torch.equal(out[33:38, 1:], x[20:])
    mask = torch.ones(40, dtype=torch.bool)
    mask[10:30] = mask[33:38] = False
    assert (out[mask] == 7.0).all()
    s.kv.read(s.cache, s.table, s.lens, torch.tensor([10, 0, 36], dtype=torch.int32, device="cuda"), out[:, :1], out[:, 1:])
    with pytest.raises(stepq.StepqError, match="out of range"):       # row 40 of 40
        s.kv.check()
    assert torch.equal(out[36:40, 1:], x[20:24]) and (whole[40:] == 7.0).all()


def test_refusals(stepq):
    s = Seqs(stepq, [20, 5], 8, 2, 64, 16)
    k = _randn(26, 25, 2, 64)
    q = _randn(27, 2, 1, 4, 64)
    o, ws = torch.empty_like(q), torch.empty(s.kv.attend_workspace_bytes(2, 1, 4, s.max_pages), dtype=torch.uint8, device="cuda")
    calls = [
        lambda: s.kv.append(s.cache, k.double(), k, s.places), lambda: s.kv.append(s.cache, k, k.half(), s.places),
        lambda: s.kv.append(s.cache, k, k, s.places.int()), lambda: s.kv.append(s.cache, k, k, s.places[:3]),
        lambda: s.kv.append(s.cache[:-1], k, k, s.places), lambda: s.kv.append(s.cache, k[:, :1], k[:, :1], s.places),
        lambda: s.kv.append(s.cache.cpu(), k, k, s.places),
        lambda: s.kv.attend(s.cache, q[:, :, :3], s.table, s.lens, 1.0, o[:, :, :3], ws),
        lambda: s.kv.attend(s.cache, q, s.table[:1], s.lens, 1.0, o, ws), lambda: s.kv.attend(s.cache, q, s.table, s.lens, 0.0, o, ws),
        lambda: s.kv.attend(s.cache, q, s.table, s.lens, float("nan"), o, ws),
        lambda: s.kv.attend(s.cache, q, s.table, s.lens, 1.0, o.half(), ws),
        lambda: s.kv.attend(s.cache, q, s.table.long(), s.lens, 1.0, o, ws),
        lambda: s.kv.attend(s.cache, q, s.table, s.lens, 1.0, o, ws[:0]),
        lambda: s.kv.read(s.cache, s.table, s.lens, s.cu[:1], k, k), lambda: s.kv.read(s.cache, s.table, s.lens, s.cu, k, k.half()),
    ]
    for i, call in enumerate(calls):
        with pytest.raises(stepq.StepqError) as e:
            call()
        assert e.value.code == stepq.EINVAL, i


def test_captured(stepq):
    """append and attend in one graph, replayed on new rows, on a stream of their own."""
    s = Seqs(stepq, [300, 40], 8, 2, 128, 16)
    k, v = _randn(28, 340, 2, 128), _randn(29, 340, 2, 128)
    s.fill(k, v)
    newest = s.places[[299, 339]].contiguous()
    k1, v1, q = k[[299, 339]].clone(), v[[299, 339]].clone(), _randn(30, 2, 1, 8, 128).bfloat16()
    o = torch.empty_like(q)
    ws = torch.empty(s.kv.attend_workspace_bytes(2, 1, 8, s.max_pages), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.kv.append(s.cache, k1, v1, newest)
        s.kv.attend(s.cache, q, s.table, s.lens, 128 ** -0.5, o, ws)
    k1.copy_(_randn(31, 2, 2, 128))
    v1.copy_(_randn(32, 2, 2, 128))
    graph.replay()
    k[[299, 339]], v[[299, 339]] = k1, v1
    _check_attend(s, q, o, None, k, v, 128 ** -0.5)


def _exact_rows(s, q, k, v, i, t, scale):
    """Sequence i, query token t, from the values that the cache holds in 64 bits: softmax weights, value rows, output and
    the bound of a score's error."""
    kd, vd = (r.double().unsqueeze(-1) * z.double() for z, r in (_quantise(x, s.bits) for x in (k, v)))
    m = s.lens_list[i] - q.shape[1] + 1 + t
    sl, rep = slice(s.cu_list[i], s.cu_list[i] + m), q.shape[2] // s.H
    kk, vv = (x[sl].repeat_interleave(rep, 1) for x in (kd, vd))
    qq = q[i, t].double()
    sc = torch.einsum("hd,mhd->hm", qq, kk) * scale
    p = torch.softmax(sc, -1)
    ds = scale * (q.shape[3] + 2) * 2.0 ** -23 * torch.einsum("hd,mhd->hm", qq.abs(), kk.abs()).amax(-1)
    return p, vv, torch.einsum("hm,mhd->hd", p, vv), ds + 2.0 ** -22 + 2.0 ** -23 * sc.abs().amax(-1)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("dtype, size", [("fp32", 1e-3), ("fp32", 1e-7), ("fp16", 1e-3), ("bf16", 1e-7)])
@pytest.mark.parametrize("sink", [False, True])
def test_attend_zero_value_rows(stepq, bits, dtype, size, sink):
    """Value rows of zeros (padding, a first token that only takes weight) add nothing, and take no bits from the others.
    A weight's error is that of its type, or 2^-25 of the largest weight times scale among the rows that are not zero."""
    d, lens = 64, [130, 70]
    s = Seqs(stepq, lens, bits, 2, d, 16)
    k, v = _randn(50, s.total, 2, d), _randn(51, s.total, 2, d) * size
    zero = [0, 17, 63, 130, 131]
    v[zero] = 0.0
    base = _randn(52, 1, 1, 2, d)
    q = (base.repeat_interleave(2, 2) + 0.01 * _randn(53, 2, 1, 4, d)).to(TYPES[dtype])
    if sink:                                             # about 18 in base 2 above the other scores
        k[[0, 130]] = base[0] * (12.5 * d ** 0.5 / base[0].square().sum(-1, keepdim=True))
    s.fill(k, v)
    got = s.read(torch.float32)[1]
    assert (got[zero] == 0).all()
    o, l = _attend(s, q)
    _check_attend(s, q, o, l, k, v, d ** -0.5)
    wt = 2.0 ** -22 if dtype == "fp32" else 2.0 ** -11
    rv = _quantise(v, bits)[1].double()
    rv[zero] = 0.0
    for i in range(2):
        p, vv, ref, ds = _exact_rows(s, q, k, v, i, 0, d ** -0.5)
        m = p.shape[1]
        r = rv[s.cu_list[i]:s.cu_list[i] + m].repeat_interleave(2, 1)
        mean = torch.einsum("hm,mhd->hd", p, vv.abs())
        floor = m * 2.0 ** -25 * (2 ** (bits - 1) - 1) * (p.transpose(0, 1) * r).amax(0)
        bound = (2 * torch.expm1(ds).unsqueeze(-1) + wt + m * 2.0 ** -23) * mean + floor.unsqueeze(-1)
        bound = bound + torch.finfo(TYPES[dtype]).eps / 2 * (ref.abs() + bound) + 2.0 ** -25 * (dtype == "fp16")
        err = (o[i, 0].double() - ref).abs()
        assert (err <= bound).all(), (i, (err / bound).max().item())


def test_attend_many_small_weights_beside_a_large_one(stepq):
    """fp32 queries: 8,191 tokens of 2^-25.5 of the first one's weight each, all in one block's share.  The scores are single
    products; a warp adds 128 tiles, the block 4 warps.  |do| <= sum p |v - o| 2 (e^ds - 1) + (weights 2^-22, sums) sum p |v|."""
    n, d, H, copies = 8192, 64, 8, 64
    s = Seqs(stepq, [n], 8, H, d, 64)
    k, v = torch.zeros(n, H, d, device="cuda"), torch.full((n, H, d), -1.0, device="cuda")
    k[0, :, 0] = 1.0
    k[1:, :, 1] = 1.0
    v[0] = 1.0
    s.fill(k, v)
    s.table, s.lens, s.max_pages = s.table.expand(copies, -1).contiguous(), s.lens.expand(copies).contiguous(), s.table.shape[1]
    q = torch.zeros(copies, 1, H, d, device="cuda")
    q[..., 0] = 25.5 * math.log(2.0) * d ** 0.5
    o, _ = _attend(s, q)
    p, vv, ref, ds = _exact_rows(s, q, k, v, 0, 0, d ** -0.5)
    away = torch.einsum("hm,mhd->hd", p, (vv - ref).abs())
    bound = 2 * torch.expm1(ds).unsqueeze(-1) * away + (2.0 ** -22 + (128 + 4 + 2) * 2.0 ** -24) * torch.einsum("hm,mhd->hd", p, vv.abs())
    err = (o[:, 0].double() - ref).abs()
    assert (err <= bound).all(), (err.max().item(), bound.max().item())


@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
def test_attend_query_channel_that_stands_out(stepq, dtype):
    """One channel of q is 2^14 times the others and meets keys that are 0 there: the others' products count in full."""
    n, d = 300, 64
    s = Seqs(stepq, [n], 8, 1, d, 32)
    k, v = _randn(54, n, 1, d), _randn(55, n, 1, d)
    k[..., 5] = 0.0
    s.fill(k, v)
    q = _randn(56, 1, 1, 4, d) * 2
    q[..., 5] = 2.0 ** 14
    q = q.to(TYPES[dtype])
    o, l = _attend(s, q)
    p, vv, ref, ds = _exact_rows(s, q, k, v, 0, 0, d ** -0.5)
    wt = 2.0 ** -22 if dtype == "fp32" else 2.0 ** -11
    mean = torch.einsum("hm,mhd->hd", p, vv.abs())
    bound = (2 * torch.expm1(ds).unsqueeze(-1) + wt + n * 2.0 ** -23) * mean
    bound = bound + torch.finfo(TYPES[dtype]).eps / 2 * (ref.abs() + bound) + 2.0 ** -25 * (dtype == "fp16")
    err = (o[0, 0].double() - ref).abs()
    assert (err <= bound).all(), (err / bound).max().item()


@pytest.mark.parametrize("bits, d, page", [(8, 128, 64), (4, 64, 16), (8, 256, 32)])
def test_attend_copy_wait_that_runs_out(stepq, bits, d, page):
    """Every stage waits for 16 bytes that never arrive: the call ends and is reported, and later calls give what they gave."""
    lens = [20000, 3000, 64, 5, 0]
    s = Seqs(stepq, lens, bits, 2, d, page)
    k, v = _randn(58, s.total, 2, d), _randn(59, s.total, 2, d)
    s.fill(k, v)
    q = _randn(60, len(lens), 2, 8, d).bfloat16()
    good, lgood = _attend(s, q)
    s.kv.set_wait_limit(4096, 16)
    with pytest.raises(stepq.StepqError, match="copy wait gave up") as e:
        _attend(s, q)
    assert e.value.code == stepq.EDEVICE
    s.kv.set_wait_limit()
    again, l = _attend(s, q)
    assert torch.equal(good, again) and torch.equal(lgood, l)


def test_check_waits_for_its_own_stream_alone(stepq):
    """A check on one stream neither waits for the default stream's work nor leaves anything to be done behind it: a bad place
    is reported by the next check, however soon it was found."""
    import gc
    gc.collect()                                         # a handle freed below would wait for the device
    s = Seqs(stepq, [16], 8, 1, 64, 16)
    k = _randn(57, 16, 1, 64)
    bad = torch.full((16,), -2, dtype=torch.int64, device="cuda")
    side, end = torch.cuda.Stream(), torch.cuda.Event()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        s.kv.append(s.cache, k, k, bad)                  # (what the first call sets up is in place)
        with pytest.raises(stepq.StepqError, match="out of range"):
            s.kv.check()
    torch.cuda._sleep(4_000_000_000)                     # two seconds on the default stream
    end.record()
    with torch.cuda.stream(side):
        for _ in range(500):
            s.kv.append(s.cache, k, k, bad)
            with pytest.raises(stepq.StepqError, match="out of range"):
                s.kv.check()
        s.kv.check()
        assert not end.query()
    torch.cuda.synchronize()


def test_attend_log_sum_of_zero_value_rows(stepq):
    """One token with a value row of zeros: o = 0, and the logarithm of the sum is its score.  The score less the reference is
    near 60 and rounded twice (2^-19 each in base 2)."""
    n, d = 64, 64
    s = Seqs(stepq, [1] * n, 8, 1, d, 16)
    k, v = _randn(61, n, 1, d), torch.zeros(n, 1, d, device="cuda")
    s.fill(k, v)
    q = _randn(62, n, 1, 4, d) * 0.05
    o, l = _attend(s, q)
    z, r = _quantise(k, 8)
    kd = r.double().unsqueeze(-1) * z.double()
    ref = torch.einsum("sihd,sd->sih", q.double(), kd[:, 0]) * d ** -0.5
    ds = d ** -0.5 * (d + 2) * 2.0 ** -23 * torch.einsum("sihd,sd->sih", q.double().abs(), kd[:, 0].abs())
    bound = ds + 2.0 ** -22 + 2 * 2.0 ** -19 * math.log(2.0) + 2.0 ** -22 * ref.abs()
    assert (o == 0).all() and ((l.double() - ref).abs() <= bound).all()


def test_check_is_refused_in_a_capture(stepq):
    """The check raises, takes nothing into the graph, and the capture goes on."""
    s = Seqs(stepq, [20], 8, 1, 64, 16)
    k, v = _randn(63, 20, 1, 64), _randn(64, 20, 1, 64)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.fill(k, v)
        with pytest.raises(stepq.StepqError, match="captur"):
            s.kv.check()
    graph.replay()
    z, r = _quantise(k, 8)
    assert torch.equal(s.read(torch.float32)[0], r.unsqueeze(-1) * z.float())


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("size", [1e35, 1e37, 6e37])
def test_attend_values_near_the_end_of_fp32(stepq, bits, dtype, size):
    """Scores spread over 2^30: every token keeps its part of the sum, however large the values are, beside rows of ordinary ones
    and of zeros."""
    lens, d = [300, 70], 64
    s = Seqs(stepq, lens, bits, 2, d, 32)
    k, v = _randn(65, s.total, 2, d), _randn(66, s.total, 2, d).clamp(-4, 4) * size
    v[5:300:7] = _randn(67, len(range(5, 300, 7)), 2, d)
    v[6:300:7] = 0.0
    s.fill(k, v)
    q = (_randn(68, 2, 1, 4, d) * 2.5).to(TYPES[dtype])
    o, l = _attend(s, q)
    _check_attend(s, q, o, l, k, v, d ** -0.5)
    wt = 2.0 ** -22 if dtype == "fp32" else 2.0 ** -11
    for i in range(2):
        p, vv, ref, ds = _exact_rows(s, q, k, v, i, 0, d ** -0.5)
        mean = torch.einsum("hm,mhd->hd", p, vv.abs())
        bound = (2 * torch.expm1(ds).unsqueeze(-1) + wt + p.shape[1] * 2.0 ** -23) * mean
        bound = bound + torch.finfo(TYPES[dtype]).eps / 2 * (ref.abs() + bound)
        err = (o[i, 0].double() - ref).abs()
        assert (err <= bound).all(), (i, (err / bound).max().item())


def test_attend_tiny_queries_of_large_keys(stepq):
    """Queries near the lower end of fp32 and keys near its upper one: scores of order 1 keep their bits."""
    n, d = 200, 64
    s = Seqs(stepq, [n], 8, 1, d, 32)
    k, v = _randn(69, n, 1, d).clamp(-4, 4) * 2.0 ** 124, _randn(70, n, 1, d)
    s.fill(k, v)
    q = _randn(71, 1, 1, 4, d) * 2.0 ** -125
    o, l = _attend(s, q)
    _check_attend(s, q, o, l, k, v, d ** -0.5)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
def test_attend_one_token_gives_its_value_row(stepq, bits, dtype):
    """A weight that stands alone is exact in fp16: o is the value row, rounded once (2^-21 for the exponential, logarithm and
    quotient)."""
    n, d = 64, 128
    s = Seqs(stepq, [1] * n, bits, 2, d, 16)
    k, v = _randn(72, n, 2, d), _randn(73, n, 2, d)
    s.fill(k, v)
    q = _randn(74, n, 1, 4, d).to(TYPES[dtype])
    o, _ = _attend(s, q)
    z, r = _quantise(v, bits)
    ref = (r.double().unsqueeze(-1) * z.double()).repeat_interleave(2, 1).unsqueeze(1)
    bound = (torch.finfo(TYPES[dtype]).eps / 2 + 2.0 ** -21) * ref.abs()
    assert ((o.double() - ref).abs() <= bound).all()
