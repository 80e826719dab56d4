"""Page tables and cache append on the GPU against the plain references:
ragged chunks, refusals, releases, exhausted lists, in-place state, padding,
duplicates, strides and both cache types."""
from __future__ import annotations

import numpy as np
import pytest

from serving_ref import TableState, e4m3_round

pytestmark = pytest.mark.gpu


class DeviceState:
    """The same allocator state as tensors, updated in place."""

    def __init__(self, ref, max_tokens):
        import torch
        t = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
        self.kv_len, self.held, self.table = t(ref.kv_len), t(ref.held), t(ref.table)
        self.free, self.count = t(ref.free), t([ref.count])
        self.max_tokens = max_tokens

    def step(self, P, chunk, idx_map=None, advance=None, advance_add=0, out_of_place=False, stream=None):
        import torch
        import markov_draft_sampling_amd as mds
        t = lambda a: None if a is None else torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
        B = len(chunk)
        qs = torch.full((B + 1,), -9, dtype=torch.int32, device="cuda")
        seq = torch.full((B,), -9, dtype=torch.int32, device="cuda")
        pos = torch.full((self.max_tokens,), -9, dtype=torch.int64, device="cuda")
        slot = torch.full((self.max_tokens,), -9, dtype=torch.int64, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        kv, held, count = self.kv_len, self.held, self.count
        if out_of_place:
            kv, held, count = kv.clone(), held.clone(), count.clone()
        mds.kv_page_tables(self.kv_len, t(chunk), self.table, self.held, self.free, self.count, P, qs, seq, pos, slot, kv,
                           held, count, status=status, idx_map=t(idx_map), advance=t(advance),
                           advance_add=advance_add, stream=stream)
        torch.cuda.synchronize()
        self.kv_len, self.held, self.count = kv, held, count
        return dict(query_start=qs.tolist(), seq_lens=seq.tolist(), positions=pos.tolist(), slot_map=slot.tolist(),
                    status=int(status.item()))


def _same(ref, dev, r, d):
    assert r == d
    assert dev.kv_len.tolist() == ref.kv_len and dev.held.tolist() == ref.held
    assert int(dev.count.item()) == ref.count
    assert dev.table.tolist() == ref.table
    assert dev.free.tolist() == ref.free


def _pair(n_slots, max_pages, P, n_pages, max_tokens, free=None):
    rng = np.random.default_rng(n_slots * 7 + P)
    free = rng.permutation(n_pages).tolist() if free is None else free
    ref = TableState(n_slots, max_pages, P, n_pages, free)
    return ref, DeviceState(ref, max_tokens)


@pytest.mark.parametrize("B,P,max_tokens", [(1, 16, 8), (5, 16, 200), (33, 32, 900), (70, 16, 5000), (1500, 16, 20000)])
def test_a_serving_loop_of_steps(B, P, max_tokens):
    rng = np.random.default_rng(B)
    n_slots = B + 7
    ref, dev = _pair(n_slots, 24, P, n_slots * 26, max_tokens)
    live = rng.permutation(n_slots)[:B].tolist()
    chunk = [int(x) for x in rng.integers(0, 12, B)]
    for step in range(7):
        adv = None
        if step:
            adv = [int(rng.integers(0, max(1, c))) for c in chunk]
            adv = [min(a, max(0, c - 1)) for a, c in zip(adv, chunk)]
        chunk = [int(x) for x in rng.choice([0, 1, 8, 8, 8, 17], B)]
        if step == 3:
            chunk[0] = min(300, max_tokens)  # a prompt chunk
        for b in range(B):
            if step > 1 and rng.random() < 0.1:
                chunk[b] = -1
        idx = list(live)
        if B > 4 and step == 4:
            idx[2] = -1  # padding rows
            idx[4] = -5
        kw = dict(idx_map=idx, advance=adv, advance_add=1 if step else 0)
        r = ref.step(chunk, max_tokens=max_tokens, **kw)
        d = dev.step(P, chunk, out_of_place=step % 2 == 1, **kw)
        _same(ref, dev, r, d)
        chunk = [max(0, c) for c in chunk]


def test_exhausted_list_and_row_ends():
    # 5 pages for requests that want 2, 3, 1 (refused), 0 (kept), 1 (refused): counted in batch order
    ref, dev = _pair(6, 4, 16, 5, 256)
    chunk = [20, 40, 10, 0, 5]
    r = ref.step(chunk, max_tokens=256)
    d = dev.step(16, chunk)
    assert r["status"] == 32 and r["seq_lens"] == [20, 40, 0, 0, 0]
    _same(ref, dev, r, d)
    # releasing the second gives its pages back first, and the same step then fits
    chunk = [1, -1, 10, 0, 5]
    r = ref.step(chunk, max_tokens=256)
    d = dev.step(16, chunk)
    assert r["seq_lens"][2] == 10 and r["status"] == 0
    _same(ref, dev, r, d)


def test_more_pages_than_a_row_and_more_tokens_than_fit():
    ref, dev = _pair(4, 2, 16, 64, 40)
    for chunk in ([33, 5, 0, 1], [32, 3, 4, 0], [0, 0, 30, 20]):  # 33 > 2 pages; then past max_tokens
        r = ref.step(chunk, max_tokens=40)
        d = dev.step(16, chunk)
        _same(ref, dev, r, d)


def test_duplicate_and_out_of_range_slots_are_padding():
    ref, dev = _pair(8, 4, 16, 40, 64)
    kw = dict(idx_map=[3, 1, 3, 9, -1, 2])
    r = ref.step([4, 4, 4, 4, 4, 4], max_tokens=64, **kw)
    d = dev.step(16, [4, 4, 4, 4, 4, 4], **kw)
    assert r["status"] == 8 and r["query_start"] == [0, 0, 4, 4, 4, 4, 8]
    _same(ref, dev, r, d)
    kw = dict(idx_map=[1, 2, 1])  # a release named twice gives nothing back
    r = ref.step([-1, 0, -1], max_tokens=64, **kw)
    d = dev.step(16, [-1, 0, -1], **kw)
    _same(ref, dev, r, d)


def test_counts_out_of_range_are_clamped():
    import torch
    ref, dev = _pair(2, 4, 16, 10, 32)
    dev.count.fill_(99)  # more than the list: taken for 10
    dev.held[1] = 50
    d = dev.step(16, [4, 4])
    assert d["status"] & 8
    assert d["seq_lens"] == [4, 4] and int(dev.count.item()) == 9
    dev.kv_len[0] = -100
    d = dev.step(16, [1, 0])
    assert d["status"] & 8 and d["positions"][0] == 0
    torch.cuda.synchronize()


@pytest.mark.parametrize("B", [3, 300])
def test_advances_at_the_ends_of_their_range(B):
    ref, dev = _pair(B, 4, 16, 4 * B, 64)
    top = 2 ** 31 - 1
    d = dev.step(16, [1] * B, advance=[top, 0, -top - 1] + ([-1] * (B - 4) + [top] if B > 3 else []), advance_add=1)
    assert d["status"] == 8 | 32  # clamped, and no room for the first (and the last)
    assert dev.kv_len.tolist()[:3] == [top, 1, 0] and d["seq_lens"][:3] == [0, 2, 1]
    if B > 3:
        assert dev.kv_len.tolist()[-1] == top and d["seq_lens"][-1] == 0


@pytest.mark.parametrize("B", [200, 3000])
def test_the_most_state_slots(B):
    n_slots = 1 << 17
    ref, dev = _pair(n_slots, 2, 16, 4096, 3 * B)
    idx = np.random.default_rng(B).permutation(n_slots)[:B].tolist()
    idx[0], idx[7], idx[9], idx[11] = n_slots - 1, n_slots, idx[B - 1], -1
    chunk = [3 if b % 5 else 1 for b in range(B)]
    for _ in range(2):
        r = ref.step(chunk, idx_map=idx, max_tokens=3 * B)
        d = dev.step(16, chunk, idx_map=idx)
        _same(ref, dev, r, d)
        chunk = [-1 if b % 3 == 0 else c for b, c in enumerate(chunk)]


def test_tables_on_a_side_stream_and_in_a_graph():
    import torch
    import markov_draft_sampling_amd as mds
    ref, dev = _pair(9, 16, 16, 200, 64)
    chunk = [8] * 8
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    r = ref.step(chunk, max_tokens=64)
    d = dev.step(16, chunk, stream=side)
    _same(ref, dev, r, d)
    # a captured decoding step, replayed with new accepted counts: state advances in place
    B = 8
    t = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    adv, ch = t([0] * B), t(chunk)
    qs, seq = t([0] * (B + 1)), t([0] * B)
    pos, slot = torch.zeros(64, dtype=torch.int64, device="cuda"), torch.zeros(64, dtype=torch.int64, device="cuda")
    call = lambda: mds.kv_page_tables(dev.kv_len, ch, dev.table, dev.held, dev.free, dev.count, 16, qs, seq, pos,  # noqa: E731
                                      slot, dev.kv_len, dev.held, dev.count, advance=adv, advance_add=1)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    rng = np.random.default_rng(5)
    for _ in range(6):
        a = [int(x) for x in rng.integers(0, 8, B)]
        adv.copy_(t(a))
        g.replay()
        torch.cuda.synchronize()
        r = ref.step(chunk, max_tokens=64, advance=a, advance_add=1)
        assert r["slot_map"] == slot.tolist() and r["positions"] == pos.tolist() and r["seq_lens"] == seq.tolist()
        assert dev.table.tolist() == ref.table and int(dev.count.item()) == ref.count


# ---------------------------------------------------------------- append --
def _append(T, H, D, P, NP, cache, layout="nhd", seed=0, pad_rows=2, special=False):
    import torch
    import markov_draft_sampling_amd as mds
    rng = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    k = torch.randn((T, H, D + 8), generator=g).to(torch.bfloat16)
    v = (torch.randn((T, H, D + 8), generator=g) * 3).to(torch.bfloat16)
    if special and T:
        k[0, 0, :6] = torch.tensor([float("nan"), float("inf"), -float("inf"), 1e30, -1e30, 0.0])
    slots = rng.permutation(NP * P)[:T].astype(np.int64)
    slots[T - pad_rows:] = -1
    if T > 4:
        slots[1] = NP * P + 3  # past the cache: skipped and flagged
    dt = torch.bfloat16 if cache == "bf16" else torch.float8_e4m3fn
    shape = (NP, P, H, D) if layout == "nhd" else (NP, H, P, D)
    mk = lambda: torch.randn(shape, generator=g).to(dt).cuda()  # noqa: E731
    kp, vp = mk(), mk()
    if layout == "hnd":
        kp, vp = kp.transpose(1, 2), vp.transpose(1, 2)
    k0, v0 = kp.clone(), vp.clone()
    ks = vs = None
    if cache == "e4m3":
        ks = torch.tensor(rng.uniform(0.003, 0.05, H), dtype=torch.float32)
        vs = torch.tensor(rng.uniform(0.003, 0.05, H), dtype=torch.float32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kd, vd = k.cuda()[..., :D], v.cuda()[..., :D]
    mds.kv_append(kd, vd, kp, vp, torch.from_numpy(slots).cuda(), k_scale=None if ks is None else ks.cuda(),
                  v_scale=None if vs is None else vs.cuda(), status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == (16 if T > 4 else 0)
    for src, sc, got, before in ((k, ks, kp, k0), (v, vs, vp, v0)):
        want = before.float().cpu().numpy().reshape(-1, H, D).astype(np.float64) if layout == "nhd" else \
            before.contiguous().float().cpu().numpy().reshape(-1, H, D).astype(np.float64)
        have = got.contiguous().float().cpu().numpy().reshape(-1, H, D)
        for t in range(T):
            if 0 <= slots[t] < NP * P:
                x = src[t, :, :D].float().numpy()
                if sc is not None:
                    with np.errstate(all="ignore"):
                        x = e4m3_round(x / sc.numpy()[:, None])
                want[slots[t]] = x
        assert np.array_equal(have.astype(np.float64), want, equal_nan=True)


@pytest.mark.parametrize("T,H,D,P,NP", [(1, 1, 16, 16, 1), (3, 2, 64, 16, 4), (40, 3, 128, 32, 3), (257, 8, 128, 64, 9),
                                        (9, 5, 112, 1024, 1)])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_append(T, H, D, P, NP, cache):
    _append(T, H, D, P, NP, cache, seed=T, pad_rows=0 if T == 1 else 2)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_append_head_major_pages_and_special_values(cache):
    _append(20, 4, 64, 16, 5, cache, layout="hnd", seed=3, special=True)


def test_append_refuses_mismatched_tensors():
    import torch
    import markov_draft_sampling_amd as mds
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
    slot = torch.zeros(4, dtype=torch.int64, device="cuda")
    kp = z(2, 16, 2, 64)
    with pytest.raises(mds.MdsError):
        mds.kv_append(z(4, 2, 32), z(4, 2, 32), kp, kp.clone(), slot)
    with pytest.raises(mds.MdsError):
        mds.kv_append(z(4, 2, 64, dt=torch.float16), z(4, 2, 64), kp, kp.clone(), slot)
    with pytest.raises(mds.MdsError):
        mds.kv_append(z(4, 2, 64), z(4, 2, 64), kp, kp.clone(), slot.cpu())
    with pytest.raises(mds.MdsError):  # an 8-bit cache needs scales
        mds.kv_append(z(4, 2, 64), z(4, 2, 64), z(2, 16, 2, 64, dt=torch.float8_e4m3fn),
                      z(2, 16, 2, 64, dt=torch.float8_e4m3fn), slot)
