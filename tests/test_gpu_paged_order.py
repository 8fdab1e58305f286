"""Attention over the paged cache: what several threads, CTAs and calls do with
the same memory.  Results are compared bit for bit where only the order in
which things happen differs, and once with the definition in float64 (the
tolerances are those of test_gpu_paged.py)."""
import threading

import pytest
import torch

import tensor_transformer_layer_cube_gb300 as t
from tests.gpu_util import assert_guards_intact, device, guarded
from tests.test_gpu_paged import Case, compare

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    c = t.tp3d_create(0)
    yield c
    t.tp3d_destroy(c)


def want64(c, dropped=()):
    """oracle.paged.attention's results by torch on the GPU, for lengths that would take numpy minutes; without the keys
    at the positions ``dropped``."""
    tokens, heads, d = c.q.shape
    g = heads // c.kv_heads
    o, absum = (torch.zeros(tokens, heads, d, dtype=torch.float64, device=device()) for _ in range(2))
    lse = torch.full((tokens, heads), -torch.inf, dtype=torch.float64, device=device())
    amax = torch.zeros(tokens, heads, dtype=torch.float64, device=device())
    for b, kv in enumerate(int(x) for x in c.kv):
        q0, q1 = int(c.q_start[b]), int(c.q_start[b + 1])
        ids = torch.from_numpy(c.table[b, :-(-kv // c.page)]).to(device())
        last = kv - (q1 - q0) + torch.arange(q1 - q0, device=device())
        hidden = torch.arange(kv, device=device()) > last[:, None]
        hidden[:, [x for x in dropped if x < kv]] = True
        for i in range(heads):
            k, v = (p[ids, :, i // g].flatten(0, 1)[:kv].double() for p in (c.kp, c.vp))
            q = c.q[q0:q1, i].double()
            s = (c.scale * (q @ k.T)).masked_fill(hidden, -torch.inf)
            lse[q0:q1, i] = s.logsumexp(1)
            p = (s - lse[q0:q1, i, None]).exp()
            o[q0:q1, i], absum[q0:q1, i] = p @ v, p @ v.abs()
            amax[q0:q1, i] = c.scale * (q.abs() @ k.abs().T).masked_fill(hidden, 0).amax(1)
    return [x.cpu().numpy() for x in (o, lse, absum, amax)]


# One CTA ends up to two split items after its range: the one that its range begins in and the one that it ends in.
# Fewer than 256 rows of each pair of tiles are some token's, so the rows of the join are dealt to other threads than
# those that weigh them.  (heads, keys, rows a head): CTAs of 152 that may end both, parts of their items: 2 with 3 and
# 4; 3 with 19 and 20, joined in two levels; 15 with 7 and 7; 1 with 8 and 8
@pytest.mark.parametrize("kv,new,heads", [([8192], [200], 64), ([65536], [200], 8), ([24000], [100], 24),
                                          ([9000, 7000, 8000], [200, 130, 256], 8)])
@pytest.mark.parametrize("d", [64, 128])
def test_two_items_ended_by_one_cta(ctx, kv, new, heads, d):
    c = Case(kv, new, heads, heads, d, 64, seed=heads, v_mean=0.5)
    o, l = c.run(ctx)
    assert t.tp3d_sync_status(ctx) == 0
    compare(c, o, l, want64(c))
    # blocks of different lengths beside it hold the SMs for a while: CTAs that start late arrive last at both items
    x = torch.rand(140, 1 << 22, device=device())
    side = torch.cuda.Stream()
    for i in range(40):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            x[:1 + 19 * (i % 8)].softmax(1)
        o2, l2 = c.run(ctx)
        assert torch.equal(o.view(torch.int16), o2.view(torch.int16)) and torch.equal(l, l2)
    assert t.tp3d_sync_status(ctx) == 0


def with_bad_page(c):
    """The case's batch with one table entry outside the pool."""
    table = c.dev[2].clone()
    table[0, 1] = -1
    return t.paged_batch(c.dev[0], c.dev[1], table, c.tokens, int(max(c.new))), table


@pytest.mark.parametrize("new", [1, 200])
def test_split_work_right_after_an_error_on_its_stream(ctx, new):
    # reading the status clears the error and the counters of split items: done when the next call's CTAs count on them
    c = Case([9000], [new], 4, 4, 128, 64, seed=3)
    want, wl = c.run(ctx)
    assert t.tp3d_sync_status(ctx) == 0
    bad, table = with_bad_page(c)
    good, o, l = c.batch(), torch.empty_like(want), torch.empty_like(wl)
    junk = torch.empty_like(want)
    busy = torch.rand(64, 1 << 20, device=device())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for i in range(40):
        o.fill_(float("nan"))
        torch.cuda.synchronize()
        t.check(t.tp3d_paged_attn(ctx, c.cache, bad, c.q, junk, None, c.scale, c.ws, side))
        busy.softmax(1)  # on the legacy stream, which the side stream does not wait for
        assert t.STATUS[t.tp3d_sync_status(ctx, side)] == "TP3D_EPAGES"
        t.check(t.tp3d_paged_attn(ctx, c.cache, good, c.q, o, l, c.scale, c.ws, side))
        assert t.tp3d_sync_status(ctx, side) == 0
        assert torch.equal(o.view(torch.int16), want.view(torch.int16)) and torch.equal(l, wl)


def test_first_call_of_a_context_on_a_side_stream():
    # a new context's counters and error word are zero before its first call on a stream that waits for no other
    c = Case([9000], [200], 4, 4, 128, 64, seed=3)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(8):
        x = t.tp3d_create(0)
        got.append(c.run(x, stream=side))
        assert t.tp3d_sync_status(x, side) == 0
        t.tp3d_destroy(x)
    for o, l in got[1:]:
        assert torch.equal(o.view(torch.int16), got[0][0].view(torch.int16)) and torch.equal(l, got[0][1])


@pytest.mark.parametrize("d", [64, 128])
def test_values_that_are_not_finite_behind_pieces_of_one_query_tile(ctx, d):
    # notes of values that are not finite, in a CTA that goes on with many pieces whose second query tile is empty: the
    # first requests have two query tiles, the others one, and most have a NaN or an infinity that only some rows see
    kv, new = [260, 300, 200] + [40 + i % 50 for i in range(700)], [200, 256, 130] + [17 + i % 7 for i in range(700)]
    c = Case(kv, new, 4, 4, d, seed=21, v_mean=0.5)
    clean, cl = c.run(ctx)
    hit = torch.zeros_like(clean, dtype=torch.bool)
    for b in range(len(kv)):
        if b % 3 == 2:
            continue
        pos, head, col = kv[b] - 1 - b % 7, b % 4, (b * 5) % d
        c.vp[int(c.table[b, pos // 16]), pos % 16, head, col] = float("nan") if b % 2 else float("inf")
        hit[int(c.q_start[b]) + pos - (kv[b] - new[b]):int(c.q_start[b + 1]), head, col] = True
    for _ in range(20):
        o, l = c.run(ctx)
        assert torch.equal(l, cl) and torch.equal(o[~hit], clean[~hit]) and not bool(o[hit].isfinite().any())
    assert t.tp3d_sync_status(ctx) == 0


@pytest.mark.parametrize("d", [64, 128])
def test_mixed_steps_that_follow_each_other_at_once(ctx, d):
    # requests with one token and with many in every step, so both kernels of a call run beside each other and read what
    # the kernel before them has just written: back to back, and captured and replayed, they give what they give with
    # the stream drained between any two calls
    page, requests, heads, kv_heads, steps = 16, 24, 4, 2, 8
    new = [70 if b % 6 == 0 else 1 for b in range(requests)]
    width, tokens = -(-70 * steps // page), sum(new)
    pages = requests * width
    gen = torch.Generator(device=device()).manual_seed(d)
    fresh = torch.tensor(new, dtype=torch.int32, device=device())
    free = torch.randperm(pages, generator=gen, device=device()).int()
    x0 = torch.empty(tokens, heads, d, dtype=torch.bfloat16, device=device()).normal_(generator=gen)

    def buffers():
        k, v = (torch.zeros(pages, page, kv_heads, d, dtype=torch.bfloat16, device=device()) for _ in range(2))
        z = {"dtype": torch.int32, "device": device()}
        return {"k": k, "v": v, "cache": t.kv_cache(k, v), "table": torch.full((requests, width), -1, **z),
                "lens": torch.zeros(steps + 1, requests, **z), "left": torch.full((steps + 1, 1), pages, **z),
                "q_start": torch.zeros(requests + 1, **z), "pos": torch.zeros(tokens, **z),
                "slots": torch.zeros(tokens, dtype=torch.int64, device=device()),
                "x": torch.cat([x0[None], torch.zeros(steps, tokens, heads, d, dtype=x0.dtype, device=device())]),
                "l": torch.zeros(steps, tokens, heads, device=device())}

    def run(s, ws, drain):
        for i in range(steps):
            batch = t.paged_batch(s["q_start"], s["lens"][i + 1], s["table"], tokens, 70)
            for call in (
                    lambda: t.tp3d_paged_plan(ctx, page, requests, tokens, s["lens"][i], fresh, free, pages, s["left"][i],
                                              s["table"], width, s["q_start"], s["lens"][i + 1], s["slots"], s["pos"],
                                              s["left"][i + 1]),
                    lambda: t.tp3d_paged_store(ctx, s["cache"], s["x"][i, :, :kv_heads], s["x"][i, :, kv_heads:], s["slots"]),
                    lambda: t.tp3d_paged_attn(ctx, s["cache"], batch, s["x"][i], s["x"][i + 1], s["l"][i], 1.0, ws)):
                t.check(call())
                if drain:
                    torch.cuda.synchronize()

    def same(a, b):
        return all(torch.equal(a[n].view(torch.uint8), b[n].view(torch.uint8)) for n in ("table", "lens", "left", "x", "l"))

    want, got, blank = buffers(), buffers(), buffers()
    ws = torch.empty(t.tp3d_paged_attn_workspace_bytes(ctx, want["cache"], heads), dtype=torch.uint8, device=device())
    run(want, ws, True)
    assert t.tp3d_sync_status(ctx) == 0

    def reset():
        for n, x in blank.items():
            if isinstance(x, torch.Tensor):
                got[n].copy_(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(got, ws, False)
    for i in range(12):
        reset()
        if i % 2:
            graph.replay()
        else:
            run(got, ws, False)
        assert t.tp3d_sync_status(ctx) == 0
        assert same(got, want)


def test_plans_of_many_requests_from_several_host_threads():
    # a context and a thread each, batches that need different amounts of shared memory, at the same time
    def step(requests):
        z = {"dtype": torch.int32, "device": device()}
        fresh = torch.ones(requests, **z)
        return [16, requests, requests, torch.zeros(requests, **z), fresh, torch.arange(requests, **z), requests,
                torch.full((1,), requests, **z), torch.zeros(requests, 1, **z), 1, torch.zeros(requests + 1, **z),
                torch.zeros(requests, **z), torch.zeros(requests, dtype=torch.int64, device=device()),
                torch.zeros(requests, **z), torch.zeros(1, **z)]

    statuses = {}

    def serve(requests):
        ctx, args, stream = t.tp3d_create(0), step(requests), torch.cuda.Stream()
        torch.cuda.synchronize()
        # the C call with its arguments ready, so that the threads spend their time in it
        plan, raw = t.lib().tp3d_paged_plan, [x if isinstance(x, int) else x.data_ptr() for x in args]
        got = {plan(ctx, *raw, stream.cuda_stream) for _ in range(20000)}
        statuses[requests] = {t.STATUS[x] for x in got | {t.tp3d_sync_status(ctx, stream.cuda_stream)}}
        t.tp3d_destroy(ctx)

    threads = [threading.Thread(target=serve, args=(n,)) for n in (16384, 8000, 12000)]
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    assert statuses == {n: {"TP3D_OK"} for n in (16384, 8000, 12000)}


@pytest.mark.parametrize("kv,new,heads,kv_heads", [
    # parts of every kind: two and three to an item, many in two levels, single tokens, both kernels of a call
    ([9000, 7000], [200, 130], 8, 8), ([30000], [64], 2, 1), ([20000], [1], 16, 2), ([5000, 6000, 300], [1, 300, 1], 8, 2)])
@pytest.mark.parametrize("d", [64, 128])
def test_workspace_between_guards(ctx, kv, new, heads, kv_heads, d):
    c = Case(kv, new, heads, kv_heads, d, 64, seed=d)
    want, wl = c.run(ctx)
    whole, ws = guarded(t.tp3d_paged_attn_workspace_bytes(ctx, c.cache, heads), torch.uint8)
    o, l = torch.empty_like(want), torch.empty_like(wl)
    t.check(t.tp3d_paged_attn(ctx, c.cache, c.batch(), c.q, o, l, c.scale, ws))
    assert t.tp3d_sync_status(ctx) == 0
    assert torch.equal(o.view(torch.int16), want.view(torch.int16)) and torch.equal(l, wl)
    assert_guards_intact(whole)
