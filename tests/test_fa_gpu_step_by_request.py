"""The decode step on batches laid out by request, where some requests add fewer
tokens than others or none: the bookkeeping against one request after another,
and the four calls in a row against each request by itself."""
import numpy as np
import pytest

import step_reference as ref
from exact_io_aware_30_gb300 import fa

torch = pytest.importorskip("torch")

import decode_formula as formula

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from exact_io_aware_30_gb300 import build
    build.build()
    fa.load()
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()
    assert fa.device_error() == fa.FA_OK


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def _by_request(lens, delta, table, ring, state, bs, n):
    """Requests that add more than n are refused; the others' rows are those of one request after another."""
    delta = np.asarray(delta, np.int64)
    wide = delta > n
    # what the packed update makes of the others (a refused one's blocks are not asked for)
    kept = np.where(wide, 0, delta)
    B, M = table.shape
    want = ref.paged_update(lens, kept, table, ring, state, bs, int(np.maximum(kept, 0).sum()))
    long = np.clip(lens, 0, M * bs) + delta > M * bs
    want["status"] = np.where(wide, np.where(long, 2, 3), want["status"]).astype(np.int32)
    slot, pos, at = np.full(B * n, -1, np.int32), np.zeros(B * n, np.int32), 0
    for b in range(B):
        add = max(int(kept[b]), 0)
        slot[(b + 1) * n - add:(b + 1) * n] = want["slot_map"][at:at + add]
        pos[(b + 1) * n - add:(b + 1) * n] = want["positions"][at:at + add]
        at += add
    want["slot_map"], want["positions"] = slot, pos
    return want


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,M,bs,n", [(1, 3, 16, 1), (7, 4, 32, 3), (64, 9, 16, 1), (300, 5, 128, 5), (1025, 3, 16, 2),
                                      (2500, 2, 64, 9), (5000, 3, 16, 1)])
def test_update_by_request_against_one_after_another(B, M, bs, n, in_place):
    rng = np.random.default_rng(B + n)
    lens = rng.integers(0, M * bs + 1, B).astype(np.int32)
    have = -(-lens // bs)
    spare = int(rng.integers(0, B + 2))
    perm = rng.permutation(int(have.sum()) + spare)
    table, at = np.full((B, M), -1, np.int32), 0
    for b in range(B):
        table[b, :have[b]] = perm[at:at + have[b]]
        at += have[b]
    ring = np.full(len(perm) + 1, -7, np.int32)
    head = int(rng.integers(0, len(ring)))
    ring[(head + np.arange(spare)) % len(ring)] = perm[at:]
    state = np.array([head, spare], np.int32)
    delta = rng.integers(0, n + 1, B)
    delta[rng.random(B) < 0.2] = 0
    delta[rng.random(B) < 0.1] = n + 1 + rng.integers(0, 1 << 30)
    delta[rng.random(B) < 0.1] = -3
    delta[rng.random(B) < 0.05] = -(2 ** 31)
    want = _by_request(lens, delta, table, ring, state, bs, n)
    t, r, l, s = _i32(table), _i32(ring), _i32(lens), _i32(state)
    slot, pos = (torch.full((B * n + 5,), x, dtype=torch.int32, device="cuda") for x in (77, 78))
    kw = dict(seq_lens_out=l, ring_state_out=s) if in_place else {}
    got = fa.paged_update(l, _i32(delta), t, r, s, bs, slot_map=slot[:B * n], positions=pos[:B * n], rows_per_request=n, **kw)
    for name in ("seq_lens", "status", "slot_map", "positions", "ring_state"):
        assert np.array_equal(getattr(got, name).cpu().numpy(), want[name]), name
    assert np.array_equal(t.cpu().numpy(), want["block_table"]) and np.array_equal(r.cpu().numpy(), want["free_ring"])
    assert bool((slot[B * n:] == 77).all()) and bool((pos[B * n:] == 78).all())


def test_update_by_request_refusals():
    l, t, r, s = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (2, 8, 4, 2))
    t = t.view(2, 4)
    step = fa.paged_update(l, l.clone(), t, r, s, 16, rows_per_request=3)
    assert step.slot_map.shape == (6,) and bool((step.slot_map == -1).all())
    fa.paged_update(l, l.clone(), t, r, s, 16, rows_per_request=3, max_tokens=6)
    for bad in (lambda: fa.paged_update(l, l.clone(), t, r, s, 16, rows_per_request=3, max_tokens=5),
                lambda: fa.paged_update(l, l.clone(), t, r, s, 16, rows_per_request=0),
                lambda: fa.paged_update(l, l.clone(), t, r, s, 16, rows_per_request=-1),
                lambda: fa.paged_update(l, l.clone(), t, r, s, 16, rows_per_request=1, slot_map=r),
                lambda: fa.paged_update(l, l.clone(), t, r, s, 17, rows_per_request=1)):
        with pytest.raises(fa.FAError):
            bad()


@pytest.mark.parametrize("dtype,H,Hkv,d,bs,n", [(torch.bfloat16, 8, 2, 128, 16, 1), (torch.float16, 4, 4, 64, 32, 1),
                                                (torch.bfloat16, 4, 1, 64, 16, 3), (torch.float16, 8, 2, 128, 16, 4)])
def test_each_request_has_its_own_positions_cache_and_output(dtype, H, Hkv, d, bs, n):
    """A captured step over four requests of which the first is idle at first, others stop, finish and come
    back, and with n > 1 each adds any number up to n: a request's new rows are rotated to its own
    positions, go to its own cache and attend to that alone."""
    B, M, pool = 4, 5, 24
    g = torch.Generator(device="cuda").manual_seed(d + n)
    rng = np.random.default_rng(d + n)
    plan = fa.rope_plan(d)
    new = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    lens, table, state, delta = new(B), new(B, M) - 1, _i32([0, pool]), new(B)
    ring = torch.randperm(pool, device="cuda", generator=g).int()
    kc, vc = (torch.full((pool, Hkv, bs, d), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((pool, Hkv), float("nan"), device="cuda") for _ in range(2))
    x = torch.zeros(B, n, H + 2 * Hkv, d, dtype=dtype, device="cuda")  # tokens by request, as a projection writes them
    q, k, v = x[:, :, :H].transpose(1, 2), x[:, :, H:H + Hkv].transpose(1, 2), x[:, :, H + Hkv:]
    qr, kr = torch.zeros(B, H, n, d, dtype=dtype, device="cuda"), torch.zeros(B, n, Hkv, d, dtype=dtype, device="cuda")
    slots, pos, status = new(B * n), new(B * n), new(B)

    def one():
        fa.paged_update(lens, delta, table, ring, state, bs, seq_lens_out=lens, ring_state_out=state, slot_map=slots,
                        positions=pos, status=status, rows_per_request=n)
        fa.rope(q, k, plan, positions=pos.view(B, n), out_q=qr, out_k=kr.transpose(1, 2))
        fa.cache_append_fp8(kr.view(B * n, Hkv, d), v.reshape(B * n, Hkv, d), slots, kc, vc, ks, vs)
        return fa.decode_paged_fp8(qr, kc, vc, ks, vs, table, lens, M * bs, mask="causal")

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = one()
    torch.cuda.synchronize()
    history = [[] for _ in range(B)]  # each request's own K and V rows, rotated one by one
    for i in range(2 * bs):
        change = rng.integers(0, n + 1, B)
        change[0] = 0 if i < 5 else change[0]           # not yet begun
        change[2] = 0 if 7 <= i < 12 else change[2]     # idle
        if i == bs:
            change[1] = -10 ** 6                        # finished; its blocks go back
        if i == bs + 3 and n > 1 and len(history[3]) > 2:
            change[3] = -2                              # rejected drafts
        change = [min(int(c), M * bs - len(h)) for c, h in zip(change, history)]
        delta.copy_(_i32(change))
        x.copy_(torch.randn(x.shape, device="cuda", generator=g))
        graph.replay()
        torch.cuda.synchronize()
        assert status.tolist() == [0] * B
        for b in range(B):
            c = change[b]
            if c < 0:
                history[b] = history[b][:max(0, len(history[b]) + c)]
                continue
            first = len(history[b])
            mine = x[b:b + 1, n - c:]
            if c:
                where = torch.arange(first, first + c, dtype=torch.int32, device="cuda")
                q1, k1 = fa.rope(mine[:, :, :H].transpose(1, 2), mine[:, :, H:H + Hkv].transpose(1, 2), plan, positions=where)
                history[b] += [(k1[0, :, j], mine[0, j, H + Hkv:].clone()) for j in range(c)]
            assert int(lens[b]) == len(history[b])
            if not c or (i % 5 and i != bs + 1):
                continue
            # its new rows: the formula over its own cache, with rows rotated to its own positions
            formula.check((o[b:b + 1, :, n - c:], lse[b:b + 1, :, n - c:]), q1, kc, vc, ks, vs, table[b:b + 1], lens[b:b + 1],
                          d ** -0.5, "causal", rows=H // Hkv * n)
            for cache, scale, which in ((kc, ks, 0), (vc, vs, 1)):
                codes, s = formula._tokens(cache, scale, table[b, :-(-len(history[b]) // bs)], len(history[b]))
                want = torch.stack([h[which] for h in history[b]], 1).double()
                # half a step of e4m3, and half of 2^-9 of the scale for each growth of it
                assert bool(((codes * s[..., None] - want).abs() <= 2.0 ** -4 * want.abs() + 2.0 ** -9 * s[..., None]).all())
