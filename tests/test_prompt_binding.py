"""The prompt-side calls of the binding, which has two ways into the C ABI: the module pa_fast and Python."""
import math
import os
import sysconfig

import pytest
import torch

from paged_kv_speculative_gb300 import _build, pa_verify as pv

PAGE = 16


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()


@pytest.fixture(params=["native", "python"])
def way(request, monkeypatch):
    """Through pa_fast, which has to be there, or without it."""
    if request.param == "python":
        monkeypatch.setattr(pv, "_fast_module", False)
    else:
        assert pv._fast()
    return request.param


def setup(kv, pages=12, hkv=2, d=128, seed=0):
    """One layer's caches and one call's arguments, on the GPU."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    t, hq, i32 = 20, 4, dict(dtype=torch.int32, device="cuda")
    shape = (pages, hkv, PAGE, d)
    s = dict(kv=kv)
    for which in "kv":
        x = torch.randn(shape, device="cuda", generator=g)
        if kv == pv.KV_BF16:
            s[which + "c"], s[which + "s"] = x.to(torch.bfloat16), None
        else:
            s[which + "s"] = (x.abs().amax(-1) / 448).contiguous()
            s[which + "c"] = (x / s[which + "s"][..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    rows = lambda h: torch.randn((t, h, d), device="cuda", generator=g).to(torch.bfloat16)
    s["q"], s["k"], s["v"] = rows(hq), rows(hkv), rows(hkv)
    s["positions"] = torch.randint(-999, 999, (2, t), device="cuda", generator=g).to(torch.int32)
    s["inv_freq"] = 1e4 ** (-torch.arange(d // 2, dtype=torch.float64, device="cuda") / (d // 2))
    s["pair_axis"] = torch.arange(d // 2, **i32) % 2
    s["slots"] = torch.randperm(pages * PAGE, device="cuda", generator=g)[:t]
    s["table"] = torch.tensor([[5, 0, 11, -1], [2, 7, -1, -1]], **i32)
    s["ctx"], s["ql"] = torch.tensor([40, 19], **i32), torch.tensor([13, 7], **i32)
    s["ref"] = torch.zeros(pages, **i32)
    s["ref"][torch.tensor([5, 0, 11, 2, 7], device="cuda")] = 1
    return s


ROPE = ("q", "k", "v", "positions", "inv_freq", "pair_axis", "slots", "kc", "vc", "ks", "vs")
CHUNK = ("q", "kc", "vc", "ks", "vs", "table", "ctx", "ql")


def rope(s, **kw):
    return pv.rope_write(*[s[n] for n in ROPE], s["kv"], **kw)


def chunk(s, **kw):
    return pv.ChunkAttention(4, 2, 128, s["kv"], 12, 4, max_seqs=2)(*[s[n] for n in CHUNK], 1 / math.sqrt(128), **kw)


# ------------------------------------------------------------------ cache types
def test_cache_types_on_the_host():
    """Python's check, on host tensors (device -1)."""
    shape = (3, 2, 16, 64)
    of = lambda t: torch.zeros(shape, dtype=torch.uint8 if t.itemsize == 1 else torch.int16).view(t)
    scale = torch.ones(shape[:3])
    ok = lambda k, v, kv: pv._caches_ok(-1, of(k), of(v), scale, scale, kv, 2, 64)
    ok(torch.bfloat16, torch.bfloat16, pv.KV_BF16)
    ok(torch.uint8, torch.float8_e4m3fn, pv.KV_FP8_E4M3)
    for bad, good, kv in [(t, torch.bfloat16, pv.KV_BF16) for t in (torch.float16, torch.int16, torch.uint8)] + [
            (t, torch.uint8, pv.KV_FP8_E4M3) for t in (torch.float8_e5m2, torch.int8, torch.bfloat16)]:
        for k, v in ((bad, good), (good, bad)):
            with pytest.raises(ValueError, match="must be torch"):
                ok(k, v, kv)


@pytest.mark.gpu
@pytest.mark.parametrize("kv,other", [(pv.KV_BF16, torch.float16), (pv.KV_BF16, torch.int16), (pv.KV_FP8_E4M3, torch.float8_e5m2),
                                      (pv.KV_FP8_E4M3, torch.int8)])
def test_caches_of_another_type_of_the_same_size_are_refused(way, kv, other):
    s = setup(kv)
    for name in ("kc", "vc"):
        bad = {**s, name: s[name].view(other)}
        before = bad[name].clone()
        for call in (rope, chunk):
            with pytest.raises(ValueError, match="must be torch"):
                call(bad)
        with pytest.raises(ValueError, match="must be torch"):
            pv.PagePool([bad["kc"]], [bad["vc"]], None if s["ks"] is None else [s["ks"]], None if s["vs"] is None else [s["vs"]])
        assert torch.equal(bad[name].view(torch.uint8), before.view(torch.uint8))


@pytest.mark.gpu
def test_codes_as_float8_and_as_bytes(way):
    s = setup(pv.KV_FP8_E4M3)
    want = chunk(s)
    f8 = {**s, "kc": s["kc"].view(torch.float8_e4m3fn), "vc": s["vc"].view(torch.float8_e4m3fn)}
    assert torch.equal(chunk(f8), want)
    rope(f8)  # writes into s's caches
    pv.PagePool([f8["kc"]], [f8["vc"]], [s["ks"]], [s["vs"]])


# ------------------------------------------------------------------ streams
@pytest.mark.gpu
def test_a_new_object_on_another_stream(way):
    """A pool and a chunk attention made while their own stream is busy, on memory that held ones, and used on another stream at
    once: their workspaces have to be zeros there (a ticket that is not leaves the growing rows unserved)."""
    i32 = dict(dtype=torch.int32, device="cuda")
    s, n = setup(pv.KV_BF16), 4
    table, lens, ref = torch.zeros((n, 5000), **i32), torch.zeros(n, **i32), torch.zeros(12, **i32)
    new = torch.tensor([20, 3, 0, 33], **i32)
    need = pv.PagePool([s["kc"]], [s["vc"]]).workspace.numel()
    chunk(s)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    dirty = [torch.full((need,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
    del dirty
    torch.cuda._sleep(200_000_000)  # clocks: a tenth of a second
    pool = pv.PagePool([s["kc"]], [s["vc"]])
    src, dst = pool.resize(table, lens, ref, new, stream=side)
    side.synchronize()
    assert lens.tolist() == [20, 3, 0, 33] and ref.tolist() == [1] * 6 + [0] * 6 and src.tolist() == [-1] * n == dst.tolist()
    torch.cuda.synchronize()
    assert pool.device_errors() == 0


# ------------------------------------------------------------------ the module
def test_the_module_is_made_for_one_torch_and_apart_from_the_library(monkeypatch, tmp_path):
    path, lib = _build.fast_path(), os.path.getmtime(_build.LIB)
    assert os.path.exists(path) and path.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    monkeypatch.setattr(_build, "LIBDIR", str(tmp_path))
    assert not os.path.exists(_build.fast_path())
    _build.build()
    assert os.path.exists(_build.fast_path()) and os.path.getmtime(_build.LIB) == lib
    monkeypatch.setattr(torch, "__version__", "0.0")  # the module of another torch is not looked at
    assert _build.fast_path() != path and not os.path.exists(_build.fast_path())
    monkeypatch.setattr(pv, "_fast_module", None)
    assert pv._fast() is False


@pytest.mark.gpu
def test_out_of_memory_is_torchs_error(way):
    """Outputs of their own, with no memory for them."""
    t, i32 = 1 << 18, dict(dtype=torch.int32, device="cuda")
    s = setup(pv.KV_BF16)
    s["q"] = torch.zeros((t, 4, 128), dtype=torch.bfloat16, device="cuda")  # 256 MB
    s["k"] = s["v"] = torch.zeros((t, 2, 128), dtype=torch.bfloat16, device="cuda")
    s["positions"], s["slots"] = torch.zeros((2, t), **i32), torch.full((t,), -1, dtype=torch.int64, device="cuda")
    call = pv.ChunkAttention(4, 2, 128, pv.KV_BF16, 12, 4, max_seqs=2)
    rope(s)
    torch.cuda.empty_cache()
    torch.cuda.set_per_process_memory_fraction((torch.cuda.memory_reserved() + (1 << 24)) / torch.cuda.get_device_properties(0).total_memory)
    try:
        held = []  # what other tests left free, in pieces that an output does not fit into
        with pytest.raises(torch.OutOfMemoryError):
            while True:
                held.append(torch.empty(1 << 26, dtype=torch.uint8, device="cuda"))
        with pytest.raises(torch.OutOfMemoryError):
            rope(s)
        with pytest.raises(torch.OutOfMemoryError):
            call(*[s[n] for n in CHUNK], 1 / math.sqrt(128))
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    rope(s)


# ------------------------------------------------------------------ both ways do the same
def tables(s):
    return s["table"].clone(), s["ctx"].clone(), s["ref"].clone()


def everything(s):
    """Every call once; what they return and leave, as host values."""
    out, err = [], torch.zeros(1, dtype=torch.int32, device="cuda")
    s = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in s.items()}
    out += [rope(s), rope(s, q_out=s["q"].clone(), pairs=pv.ROPE_NEIGHBOURS, error_flags=err), err, s["kc"], s["vc"], s["ks"], s["vs"]]
    out += [chunk(s), chunk(s, out=torch.zeros_like(s["q"]))]
    pool = pv.PagePool([s["kc"]], [s["vc"]], None if s["ks"] is None else [s["ks"]], None if s["vs"] is None else [s["vs"]])
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    table, lens, ref = tables(s)
    out += [*pool.resize(table, lens, ref, i32([50, 0])), table.clone(), lens.clone(), ref.clone()]
    pool.fork(table, lens, ref, i32([0]), i32([1]))
    src, dst = pool.resize(table, lens, ref, i32([51, 53]))
    pool.copy(src, dst)
    out += [src, dst, table.clone(), lens.clone(), ref.clone(), s["kc"].clone(), s["vc"].clone()]
    pool.resize(table, lens, ref, i32([0, -1]))
    new = pool.compact(table, lens, ref)
    out += [*new, table.clone(), ref.clone()]
    in_place = pool.compact(table, lens, ref, in_place=True)
    assert in_place[0] is table and in_place[1] is ref
    pool.copy(in_place[2], in_place[3], in_place[4])
    out += [*in_place, s["kc"], s["vc"], s["ks"], s["vs"]]
    assert pool.device_errors() == 0
    return [None if t is None else t.view(torch.uint8).cpu() if t.dtype in (torch.bfloat16, torch.float8_e4m3fn) else t.cpu() for t in out]


@pytest.mark.gpu
@pytest.mark.parametrize("kv", [pv.KV_BF16, pv.KV_FP8_E4M3])
def test_both_ways_give_the_same(kv, monkeypatch):
    s = setup(kv, seed=3)
    assert pv._fast()
    native = everything(s)
    monkeypatch.setattr(pv, "_fast_module", False)
    python = everything(s)
    assert len(native) == len(python)
    for i, (a, b) in enumerate(zip(native, python)):
        assert (a is None and b is None) or torch.equal(a, b), i


@pytest.mark.gpu
@pytest.mark.parametrize("kv", [pv.KV_BF16, pv.KV_FP8_E4M3])
def test_both_ways_refuse_the_same(way, kv):
    s = setup(kv)
    fp8 = kv == pv.KV_FP8_E4M3

    def refused(call, name, bad, error=ValueError):
        with pytest.raises(error):
            call({**s, name: bad})
    for name, bad in (("q", s["q"].float()), ("q", s["q"].cpu()), ("q", s["q"][0]), ("k", s["k"][:3]), ("k", s["k"][:, :, :64]), ("v", s["v"].transpose(0, 1)),
                      ("v", s["v"][:, :1]), ("positions", s["positions"].long()), ("positions", s["positions"][:, :2].contiguous()),
                      ("positions", s["positions"].cpu()), ("positions", s["positions"][0]), ("inv_freq", s["inv_freq"].float()),
                      ("pair_axis", s["pair_axis"][:5].contiguous()), ("pair_axis", s["pair_axis"].repeat(2)[::2]), ("slots", s["slots"].int()),
                      ("slots", s["slots"][1:]), ("kc", s["kc"][:, :, :8]), ("vc", s["vc"][:3].contiguous()), ("vc", s["vc"].cpu())):
        refused(rope, name, bad)
    for name, bad in (("q", s["q"][:, :2]), ("q", s["q"].half()), ("kc", s["kc"][1:]), ("vc", s["vc"].transpose(1, 2)), ("table", s["table"].long()),
                      ("table", s["table"][:, :3].contiguous()), ("table", s["table"][:1]), ("ctx", s["ctx"].long()), ("ctx", s["ctx"].cpu()),
                      ("ql", s["ql"][:1]), ("ql", s["ql"].repeat(2)[::2])):
        refused(chunk, name, bad)
    if fp8:
        for call in (rope, chunk):
            for name in ("ks", "vs"):
                for bad in (None, s[name].double(), s[name][1:], s[name].cpu()):
                    refused(call, name, bad)
    for kw in (dict(q_out=s["q"].float()), dict(q_out=s["q"][:3]), dict(q_out=s["q"].cpu()), dict(error_flags=torch.zeros(1, dtype=torch.int64, device="cuda")),
               dict(error_flags=torch.zeros(1, dtype=torch.int32))):
        with pytest.raises(ValueError):
            rope(s, **kw)
    for bad in (s["q"][:3], s["q"].float(), s["q"].cpu(), s["q"].repeat(1, 1, 2)[..., :128]):
        with pytest.raises(ValueError):
            chunk(s, out=bad)
    with pytest.raises(pv.PaVerifyError):
        rope(s, pairs=2)
    with pytest.raises(pv.PaVerifyError):
        pv.ChunkAttention(4, 2, 128, kv, 12, 4, max_seqs=2)(*[s[n] for n in CHUNK], -1.0)
    pool = pv.PagePool([s["kc"]], [s["vc"]], [s["ks"]] if fp8 else None, [s["vs"]] if fp8 else None)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    table, lens, ref = tables(s)
    for bad in ((table.long(), lens, ref), (table, lens.long(), ref), (table, lens, ref[:3]), (table, lens[:1], ref), (table.cpu(), lens, ref),
                (table[:, ::2], lens, ref), (table[0], lens, ref)):
        for call in (lambda *t: pool.resize(*t, i32([-1, -1])), lambda *t: pool.fork(*t, i32([0]), i32([1])), pool.compact):
            with pytest.raises(ValueError):
                call(*bad)
    for call in (lambda: pool.resize(table, lens, ref, i32([1])), lambda: pool.resize(table, lens, ref, i32([1, 1]).long()),
                 lambda: pool.fork(table, lens, ref, i32([0, 0]), i32([0])), lambda: pool.fork(table, lens, ref, i32([0]).cpu(), i32([0])),
                 lambda: pool.copy(i32([0]), i32([0, 1])), lambda: pool.copy(i32([0]).long(), i32([1])), lambda: pool.copy(i32([[0]]), i32([[1]])),
                 lambda: pool.copy(i32([0]), i32([1]), i32([1, 1])), lambda: pool.copy(i32([0]), i32([1]), i32([1]).cpu())):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(pv.PaVerifyError):
        pool.fork(table, lens, ref, i32([0] * 1025), i32([1] * 1025))
    for a, b in zip((table, lens, ref), tables(s)):
        assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("kv", [pv.KV_BF16, pv.KV_FP8_E4M3])
def test_a_whole_step_in_a_graph_beside_another_stream(way, kv):
    """Resize, copy, rotary write and attention captured with torch's kernels between them and a second attention (its own workspace)
    on a stream that forks off and joins; two graphs share the workspaces. Replays do what the calls do."""
    pages, stride, t = 60, 10, 48
    s = setup(kv, pages=pages, seed=9)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(10)
    qkv = torch.randn((t, 8, 128), device="cuda", generator=g).to(torch.bfloat16)
    pool = pv.PagePool([s["kc"]], [s["vc"]], None if s["ks"] is None else [s["ks"]], None if s["vs"] is None else [s["vs"]])
    attend = [pv.ChunkAttention(4, 2, 128, kv, pages, stride, max_seqs=3) for _ in range(2)]
    start = dict(table=i32([[-1] * stride] * 3), lens=i32([0] * 3), ref=i32([0] * pages))
    now = {k: v.clone() for k, v in start.items()}
    new, ql = i32([0] * 3), i32([0] * 3)
    positions = torch.arange(t, **dict(dtype=torch.int32, device="cuda")).repeat(2, 1)
    slots = torch.zeros(t, dtype=torch.int64, device="cuda")
    caches = (s["kc"], s["vc"], s["ks"], s["vs"])
    side = torch.cuda.Stream()

    def step():
        args = now["table"], now["lens"], now["ref"]
        src, dst = pool.resize(*args, new)
        pool.copy(src, dst)
        row = torch.repeat_interleave(torch.arange(3, device="cuda"), ql.long(), output_size=t)
        first = (ql.cumsum(0) - ql).long()
        at = now["lens"][row].long() - ql[row].long() + torch.arange(t, device="cuda") - first[row]
        slots.copy_(now["table"][row, at // PAGE].long() * PAGE + at % PAGE)
        q = pv.rope_write(qkv[:, :4], qkv[:, 4:6], qkv[:, 6:], positions, s["inv_freq"], s["pair_axis"], slots, *caches, kv)
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            b = attend[1](qkv[:, 2:6], *caches, now["table"], now["lens"], ql, 0.1)
        a = attend[0](q, *caches, now["table"], now["lens"], ql, 0.09)
        main.wait_stream(side)
        return a, b, q, src, dst

    def run(lens, count, how):
        new.copy_(i32(lens))
        ql.copy_(i32(count))
        out = how()
        torch.cuda.synchronize()
        return [x.clone() for x in (*out, *now.values())]

    plan = [([40, 8, -1], [40, 8, 0]), ([56, 24, 16], [16, 16, 16]), ([57, 0, 63], [1, 0, 47]), ([105, -1, -1], [48, 0, 0])]
    want = [run(*p, step) for p in plan]
    begin = [c.clone() for c in caches if c is not None]
    graphs, outs = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for graph in graphs:
        with torch.cuda.graph(graph):
            outs.append(step())
    for k, v in start.items():
        now[k].copy_(v)
    for i, (p, w) in enumerate(zip(plan, want)):
        def replay():
            graphs[i % 2].replay()
            return outs[i % 2]
        for j, (x, y) in enumerate(zip(run(*p, replay), w)):
            assert torch.equal(x, y), (i, j)
    for c, b in zip([c for c in caches if c is not None], begin):
        assert torch.equal(c.view(torch.uint8), b.view(torch.uint8))
    assert pool.device_errors() == 0 and attend[0].device_errors() == 0 == attend[1].device_errors()
