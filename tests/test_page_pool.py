"""Page operations (fork, resize, compact, copy): refusals on the CPU, and the
CUDA kernels against a sequential model in plain Python, entry for entry."""
import ctypes
import random

import pytest
import torch

from paged_kv_speculative_gb300 import _build, pa_verify as pv

PAGE = 16


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()


def pages(n):
    return -(-n // PAGE)


class Model:
    """The operations, one row after the other. Flags: the PA_DEVERR_* bits they raise."""

    def __init__(self, num_seqs, stride, num_pages):
        self.table = [[-1] * stride for _ in range(num_seqs)]
        self.lens, self.ref, self.flags = [0] * num_seqs, [0] * num_pages, 0

    def fork(self, parents, children):
        lens = list(self.lens)
        for i, (p, c) in enumerate(zip(parents, children)):
            n = len(lens)
            if not (0 <= p < n and 0 <= c < n) or c in children[:i] or p in children or lens[c] != 0:
                self.flags |= pv.DEVERR_LENGTHS
                continue
            k = pages(lens[p])
            self.table[c][:k] = self.table[p][:k]
            self.lens[c] = lens[p]
            for page in self.table[p][:k]:
                self.ref[page] += 1

    def resize(self, new):
        stride, n = len(self.table[0]) if self.table else 0, len(self.lens)
        src, dst = [-1] * n, [-1] * n
        grow = []
        for b in range(n):
            if new[b] > stride * PAGE:
                self.flags |= pv.DEVERR_LENGTHS
            elif 0 <= new[b] < self.lens[b]:
                for page in self.table[b][pages(new[b]):pages(self.lens[b])]:
                    self.ref[page] -= 1
                self.lens[b] = new[b]
            elif new[b] > self.lens[b]:
                grow.append(b)
        holders = list(self.ref)
        free = iter([p for p, r in enumerate(self.ref) if r == 0])
        left = sum(r == 0 for r in self.ref)
        seen = {}
        for b in grow:
            old, tail, copy = self.lens[b], None, False
            if old % PAGE:
                tail = self.table[b][pages(old) - 1]
                if holders[tail] > 1:
                    rank = seen.get(tail, 0)
                    seen[tail] = rank + 1
                    copy = rank != holders[tail] - 1
            need = pages(new[b]) - pages(old) + copy
            if need > left:
                self.flags |= pv.DEVERR_NO_PAGES
                break
            left -= need
            if copy:
                page = next(free)
                src[b], dst[b] = tail, page
                self.ref[tail] -= 1
                self.ref[page] = 1
                self.table[b][pages(old) - 1] = page
            for k in range(pages(old), pages(new[b])):
                self.table[b][k] = page = next(free)
                self.ref[page] = 1
            self.lens[b] = new[b]
        return src, dst

    def compact(self):
        live = [p for p, r in enumerate(self.ref) if r > 0]
        n = len(live)
        src = [p for p in live if p >= n]
        dst = [p for p in range(n) if self.ref[p] <= 0]
        to = dict(zip(src, dst))
        for b, length in enumerate(self.lens):
            for k in range(pages(length)):
                self.table[b][k] = to.get(self.table[b][k], self.table[b][k])
        for a, b in to.items():
            self.ref[b], self.ref[a] = self.ref[a], 0
        return src, dst


# ------------------------------------------------------------------ refusals (CPU)
def fake(n=64):
    return ctypes.c_void_p(n * 4096)  # never dereferenced: the calls below are refused before any launch


@pytest.mark.parametrize("desc,status", [((-1, 4, 8), pv.ERR_INVALID), ((1, 0, 8), pv.ERR_INVALID), ((1, 4, 0), pv.ERR_INVALID),
                                         ((1025, 4, 8), pv.ERR_UNSUPPORTED), ((1, 1 << 27, 8), pv.ERR_UNSUPPORTED)])
def test_table_descs_outside_the_envelope_are_refused(desc, status):
    L, d, p = pv.lib(), pv.PagesDesc(*desc), fake()
    assert L.pa_pages_workspace_bytes(ctypes.byref(d)) == 0
    assert L.pa_pages_fork(ctypes.byref(d), p, p, p, p, p, 1, None, None) == status
    assert L.pa_pages_resize(ctypes.byref(d), p, p, p, p, p, p, None, p, 1 << 20, None) == status
    assert L.pa_pages_compact(ctypes.byref(d), p, p, p, p, p, p, p, p, None, p, 1 << 20, None) == status
    assert pv.last_error()


def test_null_pointers_small_and_misaligned_workspaces_are_refused():
    L, d, p = pv.lib(), pv.PagesDesc(2, 4, 100), fake()
    need = L.pa_pages_workspace_bytes(ctypes.byref(d))
    assert need >= 4 * 101
    for hole in range(5):
        a = [None if i == hole else p for i in range(5)]
        assert L.pa_pages_fork(ctypes.byref(d), *a, 1, None, None) == pv.ERR_INVALID
    for hole in range(6):
        a = [None if i == hole else p for i in range(6)]
        assert L.pa_pages_resize(ctypes.byref(d), *a, None, p, need, None) == pv.ERR_INVALID
    for hole in range(8):
        a = [None if i == hole else p for i in range(8)]
        assert L.pa_pages_compact(ctypes.byref(d), *a, None, p, need, None) == pv.ERR_INVALID
    assert L.pa_pages_resize(ctypes.byref(d), *[p] * 6, None, p, need - 1, None) == pv.ERR_WORKSPACE
    assert L.pa_pages_resize(ctypes.byref(d), *[p] * 6, None, ctypes.c_void_p(4096 + 4), need, None) == pv.ERR_INVALID
    assert L.pa_pages_resize(ctypes.byref(d), *[p] * 6, None, None, need, None) == pv.ERR_INVALID
    assert L.pa_pages_fork(ctypes.byref(d), p, p, p, p, p, -1, None, None) == pv.ERR_INVALID
    assert L.pa_pages_fork(ctypes.byref(d), p, p, p, p, p, 1025, None, None) == pv.ERR_UNSUPPORTED
    assert L.pa_pages_fork(None, p, p, p, p, p, 1, None, None) == pv.ERR_INVALID
    # nothing to do: no launch, so no device is needed
    assert L.pa_pages_fork(ctypes.byref(d), p, p, p, p, p, 0, None, None) == pv.OK
    empty = pv.PagesDesc(0, 4, 100)
    assert L.pa_pages_resize(ctypes.byref(empty), *[None] * 6, None, None, 0, None) == pv.OK


def test_copy_refusals():
    L, p = pv.lib(), fake()
    one = (ctypes.c_void_p * 1)(4096)

    def call(desc, src=p, dst=p, n=1, k=one, v=one, ks=None, vs=None):
        return L.pa_pages_copy(ctypes.byref(pv.PoolDesc(*desc)), src, dst, n, None, k, v, ks, vs, None, None)
    good = (8, 1, 64, pv.KV_BF16, 1)
    assert call(good, n=0) == pv.OK
    for bad in ((0, 1, 64, 0, 1), (8, 0, 64, 0, 1), (8, 1, 64, 0, 0), (8, 1, 64, 7, 1)):
        assert call(bad) == pv.ERR_INVALID
    for bad in ((8, 1, 96, 0, 1), (8, 1, 64, 0, 65)):
        assert call(bad) == pv.ERR_UNSUPPORTED
    assert call(good, n=-1) == pv.ERR_INVALID
    for kw in (dict(src=None), dict(dst=None), dict(k=None), dict(v=None)):
        assert call(good, **kw) == pv.ERR_INVALID
    assert call((8, 1, 64, pv.KV_FP8_E4M3, 1)) == pv.ERR_INVALID  # no scales
    assert call(good, k=(ctypes.c_void_p * 1)(4104)) == pv.ERR_INVALID  # misaligned
    assert call(good, k=(ctypes.c_void_p * 1)(None)) == pv.ERR_INVALID


def test_misaligned_arrays_are_refused():
    L, d, odd, p = pv.lib(), pv.PagesDesc(2, 4, 100), ctypes.c_void_p(4096 * 9 + 2), fake()
    need, one = L.pa_pages_workspace_bytes(ctypes.byref(d)), (ctypes.c_void_p * 1)(4096)
    at = lambda n, i: [odd if j == i else p for j in range(n)]
    for i in range(6):
        a = at(6, i)  # the last: error_flags
        assert L.pa_pages_fork(ctypes.byref(d), *a[:5], 1, a[5], None) == pv.ERR_INVALID
    for i in range(7):
        assert L.pa_pages_resize(ctypes.byref(d), *at(7, i), p, need, None) == pv.ERR_INVALID
    for i in range(9):
        assert L.pa_pages_compact(ctypes.byref(d), *at(9, i), p, need, None) == pv.ERR_INVALID
    for i in range(4):
        a = at(4, i)
        assert L.pa_pages_copy(ctypes.byref(pv.PoolDesc(8, 1, 64, pv.KV_BF16, 1)), a[0], a[1], 1, a[2], one, one, None, None, a[3],
                               None) == pv.ERR_INVALID


# ------------------------------------------------------------------ against the model (GPU)
def caches(num_pages, layers=1, hkv=1, d=64, fp8=False, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    shape = (num_pages, hkv, PAGE, d)
    if not fp8:
        kv = [[torch.randn(shape, device="cuda", generator=g).to(torch.bfloat16) for _ in range(layers)] for _ in range(2)]
        return kv + [None, None]
    kv = [[torch.randint(0, 256, shape, device="cuda", generator=g, dtype=torch.uint8) for _ in range(layers)] for _ in range(2)]
    return kv + [[torch.rand(shape[:3], device="cuda", generator=g) for _ in range(layers)] for _ in range(2)]


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Device:
    def __init__(self, model, pool=None):
        self.pool = pool or pv.PagePool(*caches(len(model.ref)))
        self.table, self.lens, self.ref = i32(model.table), i32(model.lens), i32(model.ref)

    def args(self):
        return self.table, self.lens, self.ref

    def same(self, model):
        assert self.lens.tolist() == model.lens
        assert self.ref.tolist() == model.ref
        assert self.table.tolist() == model.table
        assert self.pool.device_errors() == model.flags


@pytest.mark.gpu
@pytest.mark.parametrize("num_seqs,stride,num_pages,most,seed", [(1, 1, 1, 16, 0), (3, 2, 5, 32, 1), (7, 9, 40, 144, 2),
                                                                  (40, 30, 500, 200, 3), (1024, 8, 3000, 60, 4), (65, 700, 20011, 11200, 5)])
def test_random_operations_match_the_model(num_seqs, stride, num_pages, most, seed):
    rng = random.Random(seed)
    m = Model(num_seqs, stride, num_pages)
    d = Device(m)
    for step in range(12):
        kind = rng.choice(["resize", "resize", "fork", "compact"]) if step > 1 else "resize"
        if kind == "resize":
            new = [rng.choice([-1, -1, 0, rng.randint(0, most), m.lens[b] + rng.randint(0, 20)]) for b in range(num_seqs)]
            src, dst = d.pool.resize(*d.args(), i32(new))
            assert (src.tolist(), dst.tolist()) == m.resize(new)
        elif kind == "fork":
            n = rng.randint(1, min(num_seqs, 200))
            par = [rng.randint(-1, num_seqs) for _ in range(n)]
            kid = [rng.randint(-1, num_seqs) for _ in range(n)]
            d.pool.fork(*d.args(), i32(par), i32(kid))
            m.fork(par, kid)
        else:
            in_place = rng.random() < 0.5
            table, ref, src, dst, moves = d.pool.compact(*d.args(), in_place=in_place)
            a, b = m.compact()
            assert moves.tolist() == [len(a)]
            pad = [-1] * (num_pages // 2 - len(a))
            assert (src.tolist(), dst.tolist()) == (a + pad, b + pad)
            if not in_place:
                d.table, d.ref = table, ref
        d.same(m)


@pytest.mark.gpu
def test_the_last_growing_holder_keeps_a_shared_page():
    m = Model(4, 4, 16)
    d = Device(m)

    def both(new):
        src, dst = d.pool.resize(*d.args(), i32(new))
        want = m.resize(new)
        assert (src.tolist(), dst.tolist()) == want
        d.same(m)
        return want
    both([20, 0, 0, 0])
    m.fork([0, 0], [1, 3])
    d.pool.fork(*d.args(), i32([0, 0]), i32([1, 3]))
    d.same(m)
    src, dst = both([21, 21, -1, -1])  # row 3 still holds the page: both copy
    assert src[:2] == [1, 1] and m.ref[1] == 1
    both([0, 0, -1, -1])
    m.fork([3], [0])
    d.pool.fork(*d.args(), i32([3]), i32([0]))
    src, dst = both([30, -1, -1, 40])  # every holder grows: the last one keeps it
    assert src[0] >= 0 and src[3] == -1
    assert m.flags == 0


@pytest.mark.gpu
def test_growing_stops_at_the_first_row_that_does_not_fit():
    m = Model(4, 8, 6)
    d = Device(m)
    new = [33, 80, 16, 0]  # 3 pages, 5 pages (refused), 1 page (behind a refused row)
    src, dst = d.pool.resize(*d.args(), i32(new))
    assert (src.tolist(), dst.tolist()) == m.resize(new)
    assert m.lens == [33, 0, 0, 0] and m.flags == pv.DEVERR_NO_PAGES
    d.same(m)
    d.pool.device_errors(clear=True)
    assert d.pool.device_errors() == 0


@pytest.mark.gpu
def test_bad_pages_and_counts_are_flagged_and_skipped():
    m = Model(3, 4, 8)
    m.resize([40, 20, 0])
    d = Device(m)
    d.table[0, 1] = 8  # past the pool
    d.pool.resize(*d.args(), i32([0, -1, -1]))
    assert d.pool.device_errors(clear=True) == pv.DEVERR_PAGE_RANGE
    assert d.ref.tolist() == [0, 1, 0, 1, 1, 0, 0, 0]
    d.ref[3] = 0  # row 1's page, marked free
    d.pool.resize(*d.args(), i32([-1, 0, -1]))
    assert d.pool.device_errors(clear=True) == pv.DEVERR_REFS
    assert d.ref.tolist() == [0, 1, 0, 0, 0, 0, 0, 0] and d.lens.tolist() == [0, 0, 0]
    d.lens[2], d.table[2, 0] = 10, 5
    table, ref, src, dst, moves = d.pool.compact(*d.args())
    assert d.pool.device_errors(clear=True) == pv.DEVERR_REFS and table[2, 0] == 5
    d.lens[1] = 100  # more than a row holds
    d.pool.fork(*d.args(), i32([1]), i32([0]))
    d.pool.resize(*d.args(), i32([-1, 5, -1]))
    assert d.pool.device_errors() == pv.DEVERR_LENGTHS and d.lens.tolist() == [0, 100, 10]


@pytest.mark.gpu
def test_growing_on_a_page_that_counts_as_free():
    m = Model(3, 4, 8)
    m.resize([20, 20, 0])
    d = Device(m)
    d.ref[1] = 0  # row 0's last page, marked free
    d.pool.resize(*d.args(), i32([25, 40, -1]))
    assert d.pool.device_errors(clear=True) == pv.DEVERR_REFS
    assert d.lens.tolist() == [20, 40, 0] and d.table[0, :2].tolist() == [0, 1]
    assert d.table[1, :3].tolist() == [2, 3, 1] and d.ref.tolist() == [1, 1, 1, 1, 0, 0, 0, 0]


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("layers,hkv,d,num_pages,n", [(1, 1, 64, 2, 1), (3, 2, 128, 50, 20), (2, 3, 256, 30, 11), (64, 1, 64, 9, 4), (1, 8, 128, 3000, 1400)])
def test_copy_is_bit_exact(fp8, layers, hkv, d, num_pages, n):
    kv = caches(num_pages, layers, hkv, d, fp8, seed=n)
    pool = pv.PagePool(*kv)
    g = torch.Generator().manual_seed(n)
    perm = torch.randperm(num_pages, generator=g)
    src, dst = perm[:n].tolist(), perm[n:2 * n].tolist()
    dead = set(range(0, n, 3)) if n > 2 else set()
    want = [[t.clone() for t in group] if group else None for group in kv]
    for group in want:
        for t in group or ():
            for i, (a, b) in enumerate(zip(src, dst)):
                if i not in dead:
                    t[b] = t[a].clone()
    mask = lambda x, v: i32([v if i in dead else e for i, e in enumerate(x)])
    pool.copy(mask(src, -1), mask(dst, -1))
    for a, b in zip(kv, want):
        for x, y in zip(a or (), b or ()):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert pool.device_errors() == 0
    # a device count below, at and above the list's length; an out-of-range pair
    for count in (0, n // 2, n + 5):
        kv2 = [[t.clone() for t in group] if group else None for group in want]
        pool2 = pv.PagePool(*kv2)
        pool2.copy(i32(dst), i32(src), i32([count]))
        for x, y in zip(kv2[0], want[0]):
            y = y.clone()
            for a, b in list(zip(dst, src))[:count]:
                y[b] = y[a].clone()
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    pool.copy(i32([num_pages]), i32([0]))
    assert pool.device_errors() == pv.DEVERR_PAGE_RANGE


@pytest.mark.gpu
def test_copy_past_four_gigabytes():
    """Pages whose byte offsets pass 2^32, element offsets 2^31."""
    num_pages = (1 << 31) // (8 * PAGE * 128) + 40
    k, v = (torch.empty((num_pages, 8, PAGE, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    last = num_pages - 1
    k[3].normal_()
    v[last].normal_()
    pool = pv.PagePool([k], [v])
    a, b = k[3].clone(), v[last].clone()
    pool.copy(i32([3, last]), i32([last - 1, 5]))
    assert torch.equal(k[last - 1], a) and torch.equal(v[5], b)


@pytest.mark.gpu
def test_captured_and_on_another_stream():
    m = Model(6, 40, 200)
    m.resize([100, 333, 0, 0, 17, 0])
    d = Device(m)
    new, par, kid = i32([-1] * 6), i32([0, 4]), i32([2, 3])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        d.pool.resize(*d.args(), new)  # warm-up: nothing changes
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        d.pool.fork(*d.args(), par, kid)
        src, dst = d.pool.resize(*d.args(), new)
        d.pool.copy(src, dst)
    for lens in ([-1, -1, 120, 120, -1, 4], [90, 400, 0, 0, 20, 640]):
        new.copy_(i32(lens))
        graph.replay()
        m.fork([0, 4], [2, 3])
        assert (src.tolist(), dst.tolist()) == m.resize(lens)
        d.same(m)
    d.pool.fork(*d.args(), par, kid, stream=side)
    src, dst = d.pool.resize(*d.args(), i32([5, 5, 5, 5, 5, 5]), stream=side)
    d.pool.copy(src, dst, stream=side)
    side.synchronize()
    m.fork([0, 4], [2, 3])
    assert (src.tolist(), dst.tolist()) == m.resize([5] * 6)
    d.same(m)


@pytest.mark.gpu
def test_pool_arguments_are_checked():
    k, v, _, _ = caches(4)
    with pytest.raises(ValueError):
        pv.PagePool(k, v + v)
    with pytest.raises(ValueError):
        pv.PagePool(k, [v[0][:3].contiguous()])
    with pytest.raises(ValueError):
        pv.PagePool([k[0].to(torch.uint8)], [v[0].to(torch.uint8)])  # 8-bit caches without scales
    with pytest.raises(ValueError):
        pv.PagePool([k[0].transpose(1, 2)], v)
    pool = pv.PagePool(k, v)
    table, lens, ref = i32([[0, 0], [0, 0]]), i32([0, 0]), i32([0] * 4)
    for bad in ((table.long(), lens, ref), (table, lens.long(), ref), (table, lens, ref[:3]), (table, i32([0]), ref),
                (table.cpu(), lens, ref), (table[:, ::2], lens, ref)):
        with pytest.raises(ValueError):
            pool.resize(*bad, i32([-1, -1]))
    with pytest.raises(ValueError):
        pool.fork(table, lens, ref, i32([0, 0]), i32([0]))
    with pytest.raises(ValueError):
        pool.copy(i32([0]), i32([0, 1]))


@pytest.mark.gpu
def test_more_growing_rows_than_a_page_counts():
    """Three rows hold a page that counts two: the first copies it, the second keeps it, the third is refused; no page that a row
    holds counts as free."""
    m = Model(5, 4, 10)
    m.resize([20, 0, 0, 0, 7])
    m.fork([0, 0], [1, 2])
    d = Device(m)
    d.ref[1] = 2
    src, dst = d.pool.resize(*d.args(), i32([25, 40, 40, -1, 9]))
    assert d.pool.device_errors() == pv.DEVERR_REFS
    assert d.lens.tolist() == [25, 40, 20, 0, 9]
    assert (src.tolist(), dst.tolist()) == ([1, -1, -1, -1, -1], [3, -1, -1, -1, -1])
    assert d.ref.tolist() == [3, 1, 1, 1, 1, 0, 0, 0, 0, 0]
    assert d.table[:3, :3].tolist() == [[0, 3, -1], [0, 1, 4], [0, 1, -1]]
