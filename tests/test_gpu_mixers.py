"""The served-layer calls used together, as a hybrid model's step uses them: ragged prompts through the delta rule and into
packed records, keys and values into the quantised cache, then decoding from both."""
import numpy as np
import pytest

from oracle import prefill

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

H, HK, D = 4, 2, 128


@pytest.fixture(scope="module")
def stepq():
    from quantized_recurrent_state_b200 import build as qbuild
    qbuild.build()
    from quantized_recurrent_state_b200 import stepq as s
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return s


def _tokens(seed, n, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    k = r(n, HK, D)
    return dict(q=(r(n, HK, D) * D ** -0.5).to(dtype), k=(k / k.norm(dim=-1, keepdim=True)).to(dtype), v=r(n, H, D).to(dtype),
                alpha=torch.exp2(-1 / (1 + 39 * torch.rand(n, H, generator=g, device="cuda"))),
                beta=torch.rand(n, H, generator=g, device="cuda"), o=torch.zeros(n, H, D, dtype=dtype, device="cuda"))


def _int(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_prefill_then_steps_equals_one_prefill(stepq):
    """Prompt, then three drafted tokens, then one: the states and readouts of the whole sequence in one prefill.  Both
    sides are off the recurrence by at most 2^-15 sqrt(tokens) C each (see test_gpu_delta.py)."""
    ctx = stepq.Context(stepq.Plan.build_uniform(0, 1, H, D, 6), 3)
    n = 90
    x = _tokens(1, n + 4, torch.float16)
    names = ("q", "k", "v", "alpha", "beta", "o")
    S = torch.zeros(3, 1, H, D, D, device="cuda")
    fresh = torch.ones(1, dtype=torch.bool, device="cuda")
    ctx.delta_prefill(S, _int(2), _int(0, n), *(x[m][:n] for m in names), fresh=fresh)
    ctx.delta_step(S, _int(2), *(x[m][n:n + 3].unsqueeze(0) for m in names))
    ctx.delta_step(S, _int(2), *(x[m][n + 3:].unsqueeze(0) for m in names))
    o, whole = x["o"].clone(), torch.zeros(3, 1, H, D, D, device="cuda")
    ctx.delta_prefill(whole, _int(2), _int(0, n + 4), *(x[m] for m in names), fresh=fresh)
    ctx.sync()
    C = whole[2, 0].norm(dim=1).max().item() + x["v"].abs().max().item()
    bound = 2 * 2.0 ** -15 * (n + 4) ** 0.5 * C
    assert (S[2, 0] - whole[2, 0]).norm(dim=1).max().item() <= bound
    qn = x["q"].float().norm(dim=-1).max().item()
    assert ((o - x["o"]).float().abs() <= qn * (bound + 2 * 2.0 ** -13 * C) + 2.0 ** -10 * o.float().abs()).all()
    assert (S[:2] == 0).all()


def test_prompt_into_packed_records_and_decode(stepq):
    """unpack -> delta_prefill -> requant_pack -> fused decode step, with the cache of an attention layer beside it, all on
    one stream: the decode continues from the records, the attention sees the prompt and the new token."""
    lens, n = [70, 9], 2
    plan = stepq.Plan.build_uniform(0, 1, H, D, 8)
    ctx = stepq.Context(plan, n)
    pool = torch.zeros(n * plan.slot_bytes, dtype=torch.uint8, device="cuda")
    slots = _int(1, 0)
    start = torch.randn(n, 1, H, D, D, device="cuda")
    ctx.requant_pack(pool, slots, n, 0, 1, start)
    S = torch.empty(n, H, D, D, device="cuda")
    x = _tokens(2, sum(lens), torch.bfloat16)
    kv = stepq.KVCache(8, HK, D, 16, 12)
    cache = torch.zeros(kv.bytes, dtype=torch.uint8, device="cuda")
    table = _int(0, 1, 2, 3, 4, 5, 6, 7, 8, 9).view(2, 5)
    places = torch.cat([torch.arange(70), 5 * 16 + torch.arange(9)]).cuda()
    with torch.cuda.stream(ctx.main):
        ctx.unpack(pool, slots, n, 0, 1, S)
        before = S.clone()
        ctx.delta_prefill(S, None, _int(0, 70, 79), x["q"], x["k"], x["v"], x["alpha"], x["beta"], x["o"])
        ctx.requant_pack(pool, slots, n, 0, 1, S)
        packed = torch.empty_like(S)
        ctx.unpack(pool, slots, n, 0, 1, packed)
        kv.append(cache, x["k"], x["v"][:, :HK], places)
        y = _tokens(3, n, torch.float32)
        rep = lambda t: t.repeat_interleave(H // HK, dim=1).reshape(n, 1, H, D).contiguous()  # noqa: E731
        o = torch.zeros(n, 1, H, D, device="cuda")
        ctx.decode_step_fused(pool, slots, n, 0, 1, rep(y["q"]), rep(y["k"]), y["v"].unsqueeze(1).contiguous(),
                              y["alpha"].unsqueeze(1).contiguous(), y["beta"].unsqueeze(1).contiguous(), o)
        kv.append(cache, y["k"], y["v"][:, :HK], torch.tensor([70, 5 * 16 + 9], device="cuda"))
        q = torch.randn(n, 1, H, D, device="cuda")
        out = torch.empty_like(q)
        ws = torch.empty(kv.attend_workspace_bytes(n, 1, H, 5), dtype=torch.uint8, device="cuda")
        kv.attend(cache, q, table, _int(71, 10), D ** -0.5, out, ws)
        kv.check()
    ctx.sync()
    cpu = lambda t: t.detach().float().cpu().numpy()  # noqa: E731
    at = 0
    for s, m in enumerate(lens):
        for h in range(H):
            row = lambda t, hh: cpu(t[at:at + m, hh])  # noqa: E731
            _, S_ref = prefill.sequential(cpu(before[s, h]).astype(np.float64), row(x["q"], h // 2), row(x["k"], h // 2),
                                          row(x["v"], h), cpu(x["alpha"][at:at + m, h]), cpu(x["beta"][at:at + m, h]))
            assert np.abs(cpu(S[s, h]) - S_ref).max() <= 1e-4 * np.abs(S_ref).max()
            # the decode step reads the record: one token from the unpacked state, in the tolerance of its own tests
            O_ref, _ = prefill.sequential(cpu(packed[s, h]).astype(np.float64), cpu(y["q"][s:s + 1, h // 2]), cpu(y["k"][s:s + 1, h // 2]),
                                          cpu(y["v"][s:s + 1, h]), cpu(y["alpha"][s:s + 1, h]), cpu(y["beta"][s:s + 1, h]))
            assert np.all(np.abs(cpu(o[s, 0, h]) - O_ref[0]) <= 1e-5 + 1e-4 * np.abs(O_ref).max())
            # attention over prompt and new token: 8-bit rows are off by at most r / 2, r = max |x| / 127, in keys and values
            kk = torch.cat([x["k"][at:at + m, h // 2].float(), y["k"][s:s + 1, h // 2]]).double()
            vv = torch.cat([x["v"][at:at + m, h // 2].float(), y["v"][s:s + 1, h // 2]]).double()
            p = torch.softmax(kk @ q[s, 0, h].double() * D ** -0.5, 0)
            ds = D ** -0.5 * q[s, 0, h].abs().sum().item() * kk.abs().max().item() / 254 + 1e-5
            bound = vv.abs().max().item() * (1 / 254 + 2 * (np.exp(ds) - 1)) + 1e-5
            assert ((out[s, 0, h].double() - p @ vv).abs().max().item()) <= bound
        at += m


def test_two_caches_and_contexts_at_once(stepq):
    """Calls of two handles on two streams, overlapping: each gives what it gives alone."""
    res = []
    for parallel in (False, True):
        torch.manual_seed(5)
        jobs = []
        for j in range(2):
            kv = stepq.KVCache(8, 2, 64, 16, 400)
            cache = torch.zeros(kv.bytes, dtype=torch.uint8, device="cuda")
            k, v = torch.randn(6000, 2, 64, device="cuda"), torch.randn(6000, 2, 64, device="cuda")
            table = torch.arange(375, dtype=torch.int32, device="cuda").view(1, 375)
            q = torch.randn(1, 1, 8, 64, device="cuda")
            ws = torch.empty(kv.attend_workspace_bytes(1, 1, 8, 375), dtype=torch.uint8, device="cuda")
            ctx = stepq.Context(stepq.Plan.build_uniform(0, 1, H, D, 6), 1)
            x = _tokens(7 + j, 600, torch.bfloat16)
            S = torch.zeros(1, H, D, D, device="cuda")
            jobs.append((kv, cache, k, v, torch.arange(6000, device="cuda"), table, q, torch.empty_like(q), ws, ctx, x, S,
                         torch.cuda.Stream()))
        torch.cuda.synchronize()
        for kv, cache, k, v, places, table, q, o, ws, ctx, x, S, st in jobs:
            with torch.cuda.stream(st):
                kv.append(cache, k, v, places)
                kv.attend(cache, q, table, _int(6000), 0.125, o, ws)
                ctx.delta_prefill(S, None, _int(0, 600), x["q"], x["k"], x["v"], x["alpha"], x["beta"], x["o"])
            if not parallel:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        for job in jobs:
            job[0].check()
            job[9].sync()
        res.append([t.clone() for job in jobs for t in (job[7], job[10]["o"], job[11])])
    for a, b in zip(*res):
        assert torch.equal(a, b)


def test_one_context_from_two_threads(stepq):
    """Two host threads with a stream each step states of their own through one context: what a thread enqueues before its
    call is seen by it, whatever the other does in between."""
    import threading
    ctx = stepq.Context(stepq.Plan.build_uniform(0, 1, H, D, 6), 1)
    steps = 150

    def run(parallel):
        S = [torch.zeros(2, H, D, D, device="cuda") for _ in range(2)]
        x = [_tokens(20 + j, 2, torch.float32) for j in range(2)]
        out = [torch.zeros(steps, 2, 1, H, D, device="cuda") for _ in range(2)]
        torch.cuda.synchronize()

        def work(j):
            with torch.cuda.stream(torch.cuda.Stream()):
                y = {n: t.unsqueeze(1) for n, t in x[j].items() if n in "qkv"}
                for i in range(steps):
                    y["v"].mul_(-0.9375).add_(0.125 * j)
                    ctx.delta_step(S[j], None, y["q"], y["k"], y["v"], x[j]["alpha"], x[j]["beta"], out[j][i])
                torch.cuda.current_stream().synchronize()

        threads = [threading.Thread(target=work, args=(j,)) for j in range(2)]
        for t in threads:
            t.start()
            if not parallel:
                t.join()
        for t in threads:
            t.join()
        ctx.sync()
        return S + out

    for a, b in zip(run(False), run(True)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("timing", [False, True])
def test_launches_of_four_threads_are_all_counted(stepq, timing):
    """Steps and prompts of four host threads through one context, timed or not: every launch is counted, every timed one
    reported, while another thread asks for the times."""
    import threading
    ctx = stepq.Context(stepq.Plan.build_uniform(0, 1, H, D, 6), 1)
    steps, names = 400, ("q", "k", "v", "alpha", "beta", "o")
    S = [torch.zeros(1, H, D, D, device="cuda") for _ in range(4)]
    x = [_tokens(30 + j, 20, torch.bfloat16) for j in range(4)]
    cu, seen, errors = _int(0, 20), [0], []
    torch.cuda.synchronize()
    ctx.set_timing(timing)

    def collect():
        seen[0] += sum(n for _, n in ctx.kernel_stats().values())

    def work(j):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for i in range(steps):
                    if i % 2:
                        ctx.delta_prefill(S[j], None, cu, *(x[j][n] for n in names))
                    else:
                        ctx.delta_step(S[j], None, *(x[j][n][:1].unsqueeze(0) for n in names))
        except Exception as e:
            errors.append(e)

    threads = [threading.Thread(target=work, args=(j,)) for j in range(4)]
    for t in threads:
        t.start()
    while any(t.is_alive() for t in threads):
        collect()
    for t in threads:
        t.join()
    collect()
    ctx.sync()
    assert not errors and ctx.launches == 4 * steps and seen[0] == (4 * steps if timing else 0)


def test_sync_waits_for_its_own_streams_alone(stepq):
    """sync neither waits for the default stream's work nor leaves anything to be done behind it: a bad slot is reported by the
    next one, however soon it was found."""
    import gc
    gc.collect()                                         # a handle freed below would wait for the device
    ctx = stepq.Context(stepq.Plan.build_uniform(0, 1, H, D, 6), 1)
    x = _tokens(40, 1, torch.bfloat16)
    pool, bad = torch.zeros(1, 1, H, D, D, device="cuda"), _int(3)
    side, end = torch.cuda.Stream(), torch.cuda.Event()
    torch.cuda.synchronize()

    def step():
        ctx.delta_step(pool, bad, *(x[n].unsqueeze(1) for n in ("q", "k", "v", "alpha", "beta", "o")))
        with pytest.raises(stepq.StepqError, match="slot out of range"):
            ctx.sync()

    with torch.cuda.stream(side):
        step()                                           # (what the first call sets up is in place)
    torch.cuda._sleep(4_000_000_000)                     # two seconds on the default stream
    end.record()
    with torch.cuda.stream(side):
        for _ in range(500):
            step()
        ctx.sync()
        assert not end.query()
    torch.cuda.synchronize()
