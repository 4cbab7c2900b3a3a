"""asp_weight_evict against its definition: kept slots, moved rows, weights and summaries exactly."""

import math

import pytest
import torch

from adaptive_sparse_paged_gb300 import binding as B
from tests import guards
from tests import prompt_ref as R

pytestmark = pytest.mark.gpu


def same(x, y):
    return torch.equal(x.view(torch.int16), y.view(torch.int16))


def run(dev, tokens, Hkv, d, P, keep, recent, in_place, weights=None, seed=0, same_w=False):
    batch = R.Batch(dev, tokens, [0] * len(tokens), Hkv, Hkv, d, P, seed=seed)
    pages_out = [-(-min(t, keep) // P) for t in tokens]
    dst = batch.table.clone()
    if not in_place:  # pages of their own behind the batch's
        grow = sum(pages_out)
        for name in ("k", "v"):
            c = getattr(batch, name)
            more = torch.full((grow, Hkv, P, d), 3.0, dtype=torch.bfloat16)
            setattr(batch, name, torch.cat([c, more]))
        dst.fill_(-1)
        order = torch.randperm(grow, generator=batch.gen) + batch.n_phys
        at = 0
        for b, n in enumerate(pages_out):
            dst[b, :n] = order[at:at + n].to(torch.int32)
            at += n
        batch.n_phys += grow
    kv = batch.to_device()
    slots = batch.max_pages * P
    w = torch.rand((batch.B, Hkv, slots), generator=batch.gen) if weights is None else \
        weights(batch, slots)
    for b, t in enumerate(tokens):
        w[b, :, t:] = math.nan  # not read
    w_dev = guards.guarded_like(w.to(dev), "weights")
    w_out = w_dev if same_w else guards.guarded(w.shape, torch.float32, dev, fill=5.0, what="w_out")
    kept = guards.guarded((batch.B, Hkv, keep), torch.int32, dev, fill=-3, what="kept")
    lens = guards.guarded((batch.B,), torch.int32, dev, fill=-3, what="new_lens")
    dst_dev = batch.table_dev if in_place else dst.to(dev)
    B.asp_weight_evict(kv, w_dev, keep, recent, dst_dev, w_out, kept, lens, batch.ws)
    assert B.asp_get_device_error(batch.ws) == 0
    # the definition
    k_want, v_want = batch.k.clone(), batch.v.clone()
    summ_want = torch.zeros_like(batch.summ_dev).cpu()
    w_want = w.clone() if same_w else torch.full_like(w, 5.0)
    kept_want = torch.full_like(kept, -3).cpu()
    for b, t in enumerate(tokens):
        n = min(t, keep)
        k_rows, v_rows = batch.rows(batch.k, b), batch.rows(batch.v, b)
        for h in range(Hkv):
            ids = torch.tensor(R.evict_ids(w[b, h], t, keep, recent), dtype=torch.long)
            kept_want[b, h, :n] = ids.to(torch.int32)
            w_want[b, h, :n] = w[b, h][ids]
            i = torch.arange(n)
            pages = dst[b, i // P].long()
            k_want[pages, h, i % P] = k_rows[ids, h]
            v_want[pages, h, i % P] = v_rows[ids, h]
            for p in range(-(-n // P)):
                part = k_rows[ids, h][p * P:(p + 1) * P].float()
                summ_want[b, h, p, 0], summ_want[b, h, p, 1] = part.amin(0), part.amax(0)
    assert lens.tolist() == [min(t, keep) for t in tokens]
    assert torch.equal(kept.cpu(), kept_want), "kept"
    assert torch.equal(w_out.cpu().view(torch.int32), w_want.view(torch.int32)), "weights"
    assert same(batch.k_dev.cpu(), k_want), "k"
    assert same(batch.v_dev.cpu(), v_want), "v"
    assert torch.equal(batch.summ_dev.cpu(), summ_want), "summaries"


@pytest.mark.parametrize("Hkv,d,P", [(2, 64, 16), (8, 128, 16), (1, 128, 64), (4, 64, 32),
                                     (2, 64, 64), (2, 128, 32)])
@pytest.mark.parametrize("tokens,keep,recent", [
    ([1], 1, 0), ([300, 0, 17, 256], 100, 16), ([2049, 900, 128], 600, 600),
    ([1500, 1499], 1498, 0), ([700], 1, 1), ([130, 64], 700, 3)])
@pytest.mark.parametrize("in_place", [False, True])
def test_shapes(cuda_device, Hkv, d, P, tokens, keep, recent, in_place):
    keep = min(keep, -(-max(tokens) // P) * P)
    run(cuda_device, tokens, Hkv, d, P, keep, min(recent, keep), in_place, seed=keep,
        same_w=in_place)


@pytest.mark.parametrize("kind", ["equal", "zeros", "few values", "signed zeros", "special", "spread",
                                  "ascending", "descending"])
@pytest.mark.parametrize("T", [1000, 5000])
def test_weights_that_tie_or_stretch(cuda_device, kind, T):
    def weights(batch, slots):
        u = torch.rand((batch.B, batch.Hkv, slots), generator=batch.gen)
        if kind == "equal":
            return torch.full_like(u, 0.25)
        if kind == "zeros":
            return torch.where(u < 0.1, u, torch.zeros_like(u))
        if kind == "few values":
            return (u * 4).floor()
        if kind == "signed zeros":
            return torch.where(u < 0.5, torch.zeros_like(u), -torch.zeros_like(u))
        if kind == "special":
            w = torch.randn((batch.B, batch.Hkv, slots), generator=batch.gen)
            w[u < 0.3] = math.nan
            w[(u > 0.3) & (u < 0.4)] = math.inf
            w[(u > 0.4) & (u < 0.5)] = -math.inf
            return w
        if kind == "spread":
            return torch.exp(60 * (u - 0.5))
        line = torch.arange(slots, dtype=torch.float32).expand_as(u)
        return (line if kind == "ascending" else slots - line).contiguous()
    for in_place in (False, True):
        run(cuda_device, [T, T // 2 + 7], 2, 64, 16, T // 3, 33, in_place, weights, seed=T,
            same_w=not in_place)


def test_long_segments(cuda_device):
    run(cuda_device, [40000, 70001], 1, 64, 16, 30000, 1024, True, seed=3)
    run(cuda_device, [40000, 70001], 1, 64, 64, 39999, 5, False, seed=4)


@pytest.mark.parametrize("tokens,keep", [([20000], 9000), ([9000, 16385], 8192), ([70000], 50000),
                                         ([140000, 3], 70000)])
@pytest.mark.parametrize("in_place", [False, True])
def test_several_blocks_a_segment(cuda_device, tokens, keep, in_place):
    """Few segments: several blocks share one, in registers or reading it again."""
    def ties(batch, slots):
        u = torch.rand((batch.B, batch.Hkv, slots), generator=batch.gen)
        return torch.where(u < 0.5, (u * 20).floor(), u)
    run(cuda_device, tokens, 1, 64, 16, keep, 100, in_place, ties, seed=keep, same_w=in_place)
    run(cuda_device, tokens, 1, 64, 16, keep, keep, in_place, seed=keep + 1, same_w=not in_place)


def test_many_segments(cuda_device):
    tokens = [20 + (i * 13) % 150 for i in range(150)]
    run(cuda_device, tokens, 8, 64, 16, 64, 10, True, seed=5)


def test_bad_pages(cuda_device):
    batch = R.Batch(cuda_device, [200], [0], 2, 2, 64, 16, seed=6)
    kv = batch.to_device()
    w = torch.rand((1, 2, batch.max_pages * 16), device=cuda_device)
    kept = torch.zeros((1, 2, 100), dtype=torch.int32, device=cuda_device)
    lens = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    batch.table_dev[0, 5] = -1
    B.asp_weight_evict(kv, w, 100, 100, batch.table_dev, w, kept, lens, batch.ws)
    assert B.asp_get_device_error(batch.ws) == B.ASP_DEVERR_PAGE_RANGE
    assert kept[0, 0].tolist() == list(range(100, 200))


def test_a_copy_of_the_table_is_refused(cuda_device):
    """In place is asked for by the table itself: a copy of it would be moved out of order."""
    batch = R.Batch(cuda_device, [200], [0], 2, 2, 64, 16, seed=9)
    kv = batch.to_device()
    w = torch.rand((1, 2, batch.max_pages * 16), device=cuda_device)
    kept = torch.zeros((1, 2, 100), dtype=torch.int32, device=cuda_device)
    lens = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    batch.summ_dev.fill_(3.0)
    B.asp_weight_evict(kv, w, 100, 10, batch.table_dev.clone(), w, kept, lens, batch.ws)
    assert B.asp_get_device_error(batch.ws) == B.ASP_DEVERR_PAGE_RANGE
    assert same(batch.k_dev.cpu(), batch.k) and same(batch.v_dev.cpu(), batch.v)
    assert bool((batch.summ_dev == 3.0).all()) and bool((kept == -1).all())


def test_a_refused_request_keeps_its_length(cuda_device):
    """One request's table is a copy, the other's pages are its own: the first stays as long as
    it was, the second is cut."""
    batch = R.Batch(cuda_device, [200, 150], [0, 0], 2, 2, 64, 16, seed=12)
    for name in ("k", "v"):
        c = getattr(batch, name)
        setattr(batch, name, torch.cat([c, torch.zeros((7, 2, 16, 64), dtype=torch.bfloat16)]))
    dst = batch.table.clone()
    dst[1, :7] = torch.arange(batch.n_phys, batch.n_phys + 7)
    batch.n_phys += 7
    kv = batch.to_device()
    w = torch.rand((2, 2, batch.max_pages * 16), generator=batch.gen)
    w_dev = w.to(cuda_device)
    kept = torch.zeros((2, 2, 100), dtype=torch.int32, device=cuda_device)
    lens = torch.zeros(2, dtype=torch.int32, device=cuda_device)
    B.asp_weight_evict(kv, w_dev, 100, 10, dst.to(cuda_device), w_dev, kept, lens, batch.ws)
    assert B.asp_get_device_error(batch.ws) == B.ASP_DEVERR_PAGE_RANGE
    assert lens.tolist() == [200, 100]
    assert bool((kept[0] == -1).all()) and torch.equal(w_dev[0].cpu(), w[0])
    for h in range(2):
        assert kept[1, h].tolist() == R.evict_ids(w[1, h], 150, 100, 10)


@pytest.mark.parametrize("kind", ["shifted", "reversed", "last of one", "last of many", "none"])
@pytest.mark.parametrize("P", [16, 64])
def test_a_table_with_pages_of_its_own_is_refused(cuda_device, kind, P):
    """Any page of the request's own, wherever it stands, and however many pages there are."""
    T, keep = (5000 * P - 3, 9 * P) if kind == "last of many" else (40 * P, 20 * P - 1)
    batch = R.Batch(cuda_device, [1], [0], 1, 1, 64, P, seed=13, max_pages=-(-T // P))
    n_pages, n_new = -(-T // P), -(-keep // P)
    n_phys = n_pages + n_new + 1
    perm = torch.randperm(n_phys, generator=batch.gen).to(torch.int32)
    batch.table = perm[:n_pages][None].contiguous()
    own, dst = batch.table[0], torch.full_like(batch.table, -1)
    dst[0, :n_new] = perm[n_pages:n_pages + n_new]
    if kind == "shifted":
        dst[0, :n_new] = own[-n_new:]
    elif kind == "reversed":
        dst[0, :n_new] = own[:n_new].flip(0)
    elif kind != "none":
        dst[0, n_new - 1] = own[-1]
    batch.tokens, batch.n_phys = [T], n_phys
    gen = torch.Generator(device=cuda_device).manual_seed(3)
    k = torch.randn((n_phys, 1, P, 64), generator=gen, device=cuda_device).to(torch.bfloat16)
    batch.k, batch.v = k, k + 1
    batch.to_device()
    batch.summ_dev.fill_(3.0)
    w = torch.rand((1, 1, n_pages * P), generator=gen, device=cuda_device)
    w_out = torch.full_like(w, 5.0)
    kept = torch.zeros((1, 1, keep), dtype=torch.int32, device=cuda_device)
    lens = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    B.asp_weight_evict(batch.kv, w, keep, 10, dst.to(cuda_device), w_out, kept, lens, batch.ws)
    if kind == "none":
        assert B.asp_get_device_error(batch.ws) == 0 and lens.tolist() == [keep]
        assert kept[0, 0].tolist() == R.evict_ids(w[0, 0].cpu(), T, keep, 10)
        return
    assert B.asp_get_device_error(batch.ws) == B.ASP_DEVERR_PAGE_RANGE
    assert lens.tolist() == [T] and bool((kept == -1).all()) and bool((w_out == 5.0).all())
    assert torch.equal(batch.k_dev, k) and torch.equal(batch.v_dev, k + 1)
    assert bool((batch.summ_dev == 3.0).all())


def test_entries_that_are_no_pages_are_not_shared(cuda_device):
    """The same bad entry in both tables is a bad page, not one of the request's own."""
    batch = R.Batch(cuda_device, [200], [0], 2, 2, 64, 16, seed=14)
    for name in ("k", "v"):
        c = getattr(batch, name)
        setattr(batch, name, torch.cat([c, torch.zeros((7, 2, 16, 64), dtype=torch.bfloat16)]))
    dst = torch.full_like(batch.table, -1)
    dst[0, :7] = torch.arange(batch.n_phys, batch.n_phys + 7)
    batch.n_phys += 7
    batch.table[0, 2] = dst[0, 2] = 1 << 30
    kv = batch.to_device()
    w = torch.rand((1, 2, batch.max_pages * 16), device=cuda_device)
    kept = torch.zeros((1, 2, 100), dtype=torch.int32, device=cuda_device)
    lens = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    B.asp_weight_evict(kv, w, 100, 100, dst.to(cuda_device), w, kept, lens, batch.ws)
    assert B.asp_get_device_error(batch.ws) == B.ASP_DEVERR_PAGE_RANGE
    assert lens.tolist() == [100] and kept[0, 0].tolist() == list(range(100, 200))


@pytest.mark.parametrize("d,P", [(64, 16), (128, 16), (128, 64)])
@pytest.mark.parametrize("in_place", [False, True])
def test_summaries_of_nan_keys(cuda_device, d, P, in_place):
    """Channels that hold NaN in some rows of a page, or in all: as a bulk summary of them."""
    t, keep = 6 * P, 4 * P - 3
    n_new = -(-keep // P)
    batch = R.Batch(cuda_device, [t], [0], 2, 2, d, P, seed=10)
    rows = batch.rows(batch.k, 0).clone()
    rows[:, :, 4:8] = math.nan
    rows[::2, :, 20] = math.nan
    rows[:, 1, 60] = math.nan
    batch.put(batch.k, 0, rows)
    for name in ("k", "v"):
        c = getattr(batch, name)
        setattr(batch, name, torch.cat([c, torch.zeros((n_new, 2, P, d), dtype=torch.bfloat16)]))
    dst = torch.full((1, batch.max_pages), -1, dtype=torch.int32)
    dst[0, :n_new] = torch.arange(batch.n_phys, batch.n_phys + n_new)
    batch.n_phys += n_new
    kv = batch.to_device()
    batch.summ_dev.fill_(3.0)
    w = torch.rand((1, 2, batch.max_pages * P), generator=batch.gen).to(cuda_device)
    kept = torch.zeros((1, 2, keep), dtype=torch.int32, device=cuda_device)
    lens = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    table = batch.table_dev if in_place else dst.to(cuda_device)
    B.asp_weight_evict(kv, w, keep, 5, table, w, kept, lens, batch.ws)
    got = batch.summ_dev.clone()
    after = B.PagedKV(batch.k_dev, batch.v_dev, batch.summ_dev, table, lens, 2)
    B.asp_page_summarize(after, B.ASP_SUMMARIZE_BULK, None, None, batch.ws)
    assert B.asp_get_device_error(batch.ws) == 0
    assert torch.equal(torch.isnan(got), torch.isnan(batch.summ_dev))
    assert torch.equal(got.nan_to_num(0.5), batch.summ_dev.nan_to_num(0.5))


@pytest.mark.parametrize("P", [16, 64])
def test_a_page_without_rows_keeps_its_summary(cuda_device, P):
    """Every row of it lay in pages that are not there: nothing moved, nothing is said of it."""
    batch = R.Batch(cuda_device, [3 * P], [0], 2, 2, 64, P, seed=15)
    batch.table[0, 1] = -1
    kv = batch.to_device()
    batch.summ_dev.fill_(3.0)
    w = torch.rand((1, 2, batch.max_pages * P), device=cuda_device)
    kept = torch.zeros((1, 2, 3 * P), dtype=torch.int32, device=cuda_device)
    lens = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    B.asp_weight_evict(kv, w, 3 * P, 0, batch.table_dev, w, kept, lens, batch.ws)
    assert B.asp_get_device_error(batch.ws) == B.ASP_DEVERR_PAGE_RANGE
    assert bool((batch.summ_dev[:, :, 1] == 3.0).all())
    for p in (0, 2):
        part = batch.k[int(batch.table[0, p])].float()
        assert torch.equal(batch.summ_dev[0, :, p, 0].float().cpu(), part.amin(1))
        assert torch.equal(batch.summ_dev[0, :, p, 1].float().cpu(), part.amax(1))


def test_graph_replay(cuda_device):
    """Into other pages the call can be repeated: a graph of it, replayed, leaves the same."""
    batch = R.Batch(cuda_device, [500, 300], [0, 0], 2, 2, 64, 16, seed=7, max_pages=64)
    dst = torch.arange(batch.n_phys, batch.n_phys + 2 * 13, dtype=torch.int32)
    for name in ("k", "v"):
        c = getattr(batch, name)
        setattr(batch, name, torch.cat([c, torch.zeros((26, 2, 16, 64), dtype=torch.bfloat16)]))
    batch.n_phys += 26
    kv = batch.to_device()
    table = torch.full((2, 64), -1, dtype=torch.int32, device=cuda_device)
    table[:, :13] = dst.view(2, 13).to(cuda_device)
    w = torch.rand((2, 2, 64 * 16), device=cuda_device)
    w_out = torch.zeros_like(w)
    kept = torch.zeros((2, 2, 200), dtype=torch.int32, device=cuda_device)
    lens = torch.zeros(2, dtype=torch.int32, device=cuda_device)
    args = (kv, w, 200, 50, table, w_out, kept, lens, batch.ws)
    B.asp_weight_evict(*args)
    torch.cuda.synchronize()
    want = [t.clone() for t in (batch.k_dev, batch.v_dev, batch.summ_dev, w_out, kept, lens)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.asp_weight_evict(*args)
    for t in (w_out, kept, lens, batch.summ_dev):
        t.zero_()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    for x, y in zip(want, (batch.k_dev, batch.v_dev, batch.summ_dev, w_out, kept, lens)):
        assert torch.equal(x.nan_to_num(7), y.nan_to_num(7)) if x.is_floating_point() else torch.equal(x, y)
