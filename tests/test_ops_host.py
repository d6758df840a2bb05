"""Host-side checks of the operators of include/w4g128_ops.h that need no GPU:
their symbols, argument structs and refusals, returned before anything is
launched."""
import ctypes
import re

import pytest

import int4_weight_only_g128_gb300 as w

E_INVALID, E_SHAPE, E_ALIGN, E_WS, E_CUDA, E_DEVICE = 1, 2, 3, 4, 5, 6
FAKE = 0x10000  # aligned, non-null, never dereferenced on these paths


@pytest.fixture(scope="module")
def L():
    return w.lib()


def header():
    with open(w._INCLUDE + "/w4g128_ops.h") as f:
        return f.read()


def test_every_operator_is_exported(L):
    names = w.exported_symbols(("w4g128_ops.h",))
    assert names and "w4g128_sample" in names
    for n in names:
        assert hasattr(L, n), n
        assert hasattr(w.lib_debug(), n), n
        assert n in w.__all__, n


def test_constants_match_the_header():
    text = header()
    for name in ("MAX_SAMPLE_ROWS", "MAX_VOCAB", "MAX_SEQUENCES", "ERR_CACHE", "MAX_EXPERTS", "MAX_TOP_K"):
        assert re.search(rf"#define W4G128_{name} {getattr(w, name)}\b", text), name


def test_structs_match_the_header():
    """Field names and order of each argument struct."""
    for cls, name in ((w.SampleArgs, "w4g128_sample_args"), (w.AttendArgs, "w4g128_attend_args"),
                      (w.MoEArgs, "w4g128_moe_args")):
        body = re.search(r"typedef struct \{([^}]*)\} " + name + ";", header()).group(1)
        body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
        fields = [f.split()[-1].lstrip("*") for line in body.split(";") if line.strip()
                  for f in line.replace(",", " ,").split(",")]
        assert fields == [f[0] for f in cls._fields_], name


def sample(**kw):
    a = dict(logits=FAKE, row_stride=100, u=FAKE, tokens=FAKE, rows=1, vocab=100)
    a.update(kw)
    return w.lib().w4g128_sample(ctypes.byref(w.SampleArgs(**a)), None)


def test_sample_refusals(L):
    assert L.w4g128_sample(None, None) == E_INVALID
    assert sample(logits=None) == E_INVALID
    assert sample(u=None) == E_INVALID
    assert sample(tokens=None) == E_INVALID
    assert sample(rows=0) == E_INVALID and sample(rows=w.MAX_SAMPLE_ROWS + 1) == E_INVALID
    assert sample(vocab=0) == E_SHAPE
    assert sample(vocab=w.MAX_VOCAB + 1, row_stride=1 << 20) == E_SHAPE
    assert sample(row_stride=99) == E_SHAPE
    assert sample(logits=FAKE + 1) == E_ALIGN
    for f in ("temperature", "top_k", "top_p", "min_p", "u", "tokens", "logprobs"):
        assert sample(**{f: FAKE + 2}) == E_ALIGN, f
    with pytest.raises(w.W4G128Error) as ei:
        w.w4g128_sample(w.SampleArgs(logits=FAKE, row_stride=1, u=FAKE, tokens=FAKE, rows=1, vocab=2), stream=0)
    assert ei.value.status == E_SHAPE


def attend_args(**kw):
    a = dict(q=FAKE, k_new=FAKE, v_new=FAKE, k_cache=FAKE, v_cache=FAKE, page_table=FAKE, row_offsets=FAKE, lens=FAKE,
             out=FAKE, q_row=512, kv_row=128, out_row=512, page_stride=2048, slot_stride=128, head_stride=64,
             table_row=8, rows=4, count=1, q_heads=8, kv_heads=2, head_dim=64, pages=8, page_size=16, max_len=100,
             max_new=4, window=0, sinks=0, scale=0.125)
    a.update(kw)
    return w.AttendArgs(**a)


def attend(ws=FAKE, ws_bytes=1 << 40, **kw):
    return w.lib().w4g128_attend(ctypes.byref(attend_args(**kw)), ws, ws_bytes, None)


def test_attend_refusals(L):
    assert L.w4g128_attend(None, FAKE, 1 << 40, None) == E_INVALID
    for f in ("q", "k_new", "v_new", "k_cache", "v_cache", "page_table", "row_offsets", "lens", "out"):
        assert attend(**{f: None}) == E_INVALID, f
    assert attend(ws=None) == E_INVALID
    for kw in (dict(rows=0), dict(rows=(1 << 20) + 1), dict(count=0), dict(count=w.MAX_SEQUENCES + 1), dict(max_new=0),
               dict(max_new=17), dict(window=-1), dict(sinks=-1, window=5), dict(sinks=4),
               dict(scale=float("nan")), dict(scale=float("inf"))):
        assert attend(**kw) == E_INVALID, kw
    for kw in (dict(q_heads=7), dict(q_heads=34, q_row=4096), dict(kv_heads=0), dict(head_dim=96), dict(head_dim=32),
               dict(pages=0), dict(page_size=8), dict(page_size=24), dict(max_len=0), dict(max_len=(1 << 24) + 1),
               dict(max_len=129), dict(q_row=504), dict(out_row=504), dict(kv_row=120), dict(slot_stride=56),
               dict(head_stride=56), dict(page_stride=32)):
        assert attend(**kw) == E_SHAPE, kw
    for f in ("q", "k_new", "v_new", "k_cache", "v_cache", "out"):
        assert attend(**{f: FAKE + 8}) == E_ALIGN, f
    for f in ("page_table", "row_offsets", "lens"):
        assert attend(**{f: FAKE + 2}) == E_ALIGN, f
    for f, v in (("q_row", 516), ("kv_row", 132), ("out_row", 516), ("page_stride", 2052), ("slot_stride", 132),
                 ("head_stride", 68)):
        assert attend(**{f: v}) == E_ALIGN, f
    assert attend(ws=FAKE + 8) == E_ALIGN
    need = w.w4g128_attend_workspace_bytes(attend_args())
    assert need > 0 and attend(ws_bytes=need - 1) == E_WS
    assert w.w4g128_attend_workspace_bytes(attend_args(max_new=0)) == 0
    # the longest cache with the most rows does not overflow the query
    big = attend_args(max_len=1 << 24, count=1024, max_new=16, table_row=1 << 20, q_heads=256, q_row=1 << 15,
                      kv_heads=16, head_dim=128, slot_stride=2048, head_stride=128, page_stride=1 << 15, kv_row=2048,
                      out_row=1 << 15)
    assert w.w4g128_attend_workspace_bytes(big) > 1 << 40


def moe_args(**kw):
    a = dict(x=FAKE, residual=None, y=FAKE + 0x1000, router=FAKE, gate_up=FAKE, down=FAKE, M=2, D=256, F=128, E=4,
             top_k=2, renormalize=1)
    a.update(kw)
    return w.MoEArgs(**a)


def moe(ws=FAKE, ws_bytes=1 << 40, **kw):
    return w.lib().w4g128_moe(ctypes.byref(moe_args(**kw)), ws, ws_bytes, None)


def test_moe_refusals(L):
    assert L.w4g128_moe(None, FAKE, 1 << 40, None) == E_INVALID
    for f in ("x", "y", "router", "gate_up", "down"):
        assert moe(**{f: None}) == E_INVALID, f
    assert moe(ws=None) == E_INVALID
    for kw in (dict(M=0), dict(M=17), dict(top_k=0), dict(top_k=5), dict(top_k=17, E=32), dict(renormalize=2),
               dict(renormalize=-1), dict(y=FAKE)):
        assert moe(**kw) == E_INVALID, kw
    for kw in (dict(D=0), dict(D=192), dict(D=65536 + 128), dict(F=64), dict(F=200), dict(F=65536 + 128), dict(E=0),
               dict(E=w.MAX_EXPERTS + 1)):
        assert moe(**kw) == E_SHAPE, kw
    for f in ("x", "residual", "y", "router", "gate_up", "down"):
        assert moe(**{f: FAKE + 0x2008}) == E_ALIGN, f
    assert moe(ws=FAKE + 8) == E_ALIGN
    need = w.w4g128_moe_workspace_bytes(moe_args())
    assert need > 0 and moe(ws_bytes=need - 1) == E_WS
    assert w.w4g128_moe_workspace_bytes(moe_args(M=0)) == 0
    assert w.w4g128_moe_workspace_bytes(moe_args(M=16, D=65536, F=65536, E=512, top_k=16)) > 256 * 65536 * 6


_FAULT_CHILD = """
import ctypes, sys
sys.path[:0] = [{root!r}, {root!r} + "/tests"]
import test_ops_host as t
print(t.sample(), t.attend(), t.moe(), t.moe(M=0))
"""


@pytest.mark.parametrize("mode,status", [("launch", E_CUDA), ("workspace", E_WS)])
def test_host_fault_hook(mode, status):
    """W4G128_FAULT reaches the operators too, after their argument checks."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "-c", _FAULT_CHILD.format(root=root)], capture_output=True, text=True,
                         env=dict(os.environ, W4G128_FAULT=mode), timeout=120)
    assert out.returncode == 0, out.stderr
    assert [int(v) for v in out.stdout.split()] == [status] * 3 + [E_INVALID]


def test_tensors_are_checked_by_the_binding():
    torch = pytest.importorskip("torch")
    logits = torch.zeros(100, dtype=torch.bfloat16)
    with pytest.raises(w.W4G128Error):  # not on a GPU
        w.SampleArgs(logits=logits, row_stride=100, u=FAKE, tokens=FAKE, rows=1, vocab=100)
    with pytest.raises(TypeError):
        w.SampleArgs(logit=FAKE)


def test_no_device_is_reported():
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert sample() == E_DEVICE
    assert attend() == E_DEVICE
    assert moe() == E_DEVICE


def test_a_header_added_later_is_named(tmp_path, monkeypatch):
    """By default every public header but the operators', without a list to keep up."""
    import os
    import shutil
    for fn in os.listdir(w._INCLUDE):
        shutil.copy(os.path.join(w._INCLUDE, fn), tmp_path)
    before = w.exported_symbols()
    (tmp_path / "w4g128_later.h").write_text("W4G128_API int w4g128_later(int n);\n")
    monkeypatch.setattr(w, "_INCLUDE", str(tmp_path))
    assert sorted(w.exported_symbols()) == sorted(before + ["w4g128_later"])
    assert not set(before) & set(w.exported_symbols(("w4g128_ops.h",)))


def test_attend_refuses_a_scale_that_overflows_with_log2_e(L):
    """The scores are taken to base 2: scale log2(e) has to be a float, too."""
    for scale in (2.4e38, -2.4e38, 3.4e38):
        assert attend(scale=scale) == E_INVALID, scale
        assert w.w4g128_attend_workspace_bytes(attend_args(scale=scale)) == 0
    for scale in (2.35e38, -2.35e38, 0.0, 1e-45):
        assert w.w4g128_attend_workspace_bytes(attend_args(scale=scale)) > 0, scale


def sample_args(**kw):
    return w.SampleArgs(**{**dict(logits=FAKE, row_stride=100, u=FAKE, tokens=FAKE, rows=1, vocab=100), **kw})


class OnGpu:
    """A CPU tensor that says it is on a GPU, for the binding's checks."""
    is_cuda = True

    def __init__(self, t, index=0):
        import torch
        self._t, self.device = t, torch.device("cuda", index)

    def __getattr__(self, name):
        return getattr(self._t, name)


def gpu(*shape, dtype="float32", index=0):
    import torch
    return OnGpu(torch.zeros(shape, dtype=getattr(torch, dtype)), index)


def view(t, f):
    """A view of a tensor that says it is on a GPU."""
    return OnGpu(f(t._t), t.device.index)


def sample_tensors(**kw):
    a = dict(logits=gpu(4, 100, dtype="bfloat16"), row_stride=100, u=gpu(4), tokens=gpu(4, dtype="int32"), rows=4,
             vocab=100)
    a.update(kw)
    return w.SampleArgs(**a)


def attend_tensors(**kw):
    a = dict(q=gpu(4, 8, 64, dtype="bfloat16"), k_new=None, v_new=None, k_cache=gpu(8, 16, 2, 64, dtype="bfloat16"),
             v_cache=gpu(8, 16, 2, 64, dtype="bfloat16"), page_table=gpu(1, 8, dtype="int32"),
             row_offsets=gpu(2, dtype="int32"), lens=gpu(1, dtype="int32"), out=gpu(4, 8, 64, dtype="bfloat16"), q_row=512,
             out_row=512, page_stride=2048, slot_stride=128, head_stride=64, table_row=8, rows=4, count=1, q_heads=8,
             kv_heads=2, head_dim=64, pages=8, page_size=16, max_len=100, max_new=4, window=0, sinks=0, scale=0.125)
    a.update(kw)
    return w.AttendArgs(**a)


def moe_tensors(**kw):
    bf = lambda *s: gpu(*s, dtype="bfloat16")  # noqa: E731
    a = dict(x=bf(2, 256), residual=bf(2, 256), y=bf(2, 256), router=bf(4, 256),
             gate_up=gpu(4, w.w4g128_packed_bytes(256, 256), dtype="uint8"),
             down=gpu(4, w.w4g128_packed_bytes(128, 256), dtype="uint8"), M=2, D=256, F=128, E=4, top_k=2, renormalize=1)
    a.update(kw)
    return w.MoEArgs(**a)


def test_tensors_of_other_layouts_are_refused():
    """A field without a stride wants a contiguous tensor, one with strides neighbouring elements of a row."""
    pytest.importorskip("torch")
    sample_tensors(), attend_tensors(), moe_tensors()  # as they should be
    sample_tensors(logits=view(gpu(4, 200, dtype="bfloat16"), lambda t: t[:, :100]), row_stride=200)
    attend_tensors(k_cache=view(gpu(8, 2, 16, 64, dtype="bfloat16"), lambda t: t.transpose(1, 2)), slot_stride=64,
                   head_stride=1024)
    attend_tensors(page_table=view(gpu(1, 9, dtype="int32"), lambda t: t[:, :8]), table_row=9)
    sample_tensors(temperature=view(gpu(9), lambda t: t[3:7]))
    every_other = lambda *s, dtype="float32": view(gpu(*s, 2, dtype=dtype), lambda t: t[..., 0])  # noqa: E731
    for make, bad in ((sample_tensors, dict(u=every_other(4))),
                      (sample_tensors, dict(temperature=every_other(4))),
                      (sample_tensors, dict(top_k=every_other(4, dtype="int32"))),
                      (sample_tensors, dict(tokens=every_other(4, dtype="int32"))),
                      (sample_tensors, dict(logprobs=every_other(4))),
                      (sample_tensors, dict(logits=view(gpu(100, 4, dtype="bfloat16"), lambda t: t.t()))),
                      (attend_tensors, dict(q=every_other(4, 8, 64, dtype="bfloat16"))),
                      (attend_tensors, dict(out=every_other(4, 8, 64, dtype="bfloat16"))),
                      (attend_tensors, dict(k_cache=view(gpu(8, 16, 64, 2, dtype="bfloat16"), lambda t: t.transpose(2, 3)))),
                      (attend_tensors, dict(page_table=every_other(1, 8, dtype="int32"))),
                      (attend_tensors, dict(row_offsets=every_other(2, dtype="int32"))),
                      (moe_tensors, dict(x=view(gpu(256, 2, dtype="bfloat16"), lambda t: t.t()))),
                      (moe_tensors, dict(x=view(gpu(2, 512, dtype="bfloat16"), lambda t: t[:, :256]))),
                      (moe_tensors, dict(y=view(gpu(2, 512, dtype="bfloat16"), lambda t: t[:, :256]))),
                      (moe_tensors, dict(router=view(gpu(256, 4, dtype="bfloat16"), lambda t: t.t())))):
        with pytest.raises(w.W4G128Error) as ei:
            make(**bad)
        assert ei.value.status == E_INVALID, bad


def test_tensors_and_workspaces_of_other_devices_are_refused(monkeypatch):
    """Tensors share a device, the current one when the call is made or marshalled; a workspace is on it, too."""
    torch = pytest.importorskip("torch")
    with pytest.raises(w.W4G128Error) as ei:
        sample_tensors(u=gpu(4, index=1))
    assert ei.value.status == E_INVALID
    elsewhere = [attend_tensors()] * 2 + [moe_tensors()] * 2 + [sample_tensors()] * 2
    called, strings = [], w.lib().w4g128_status_string

    class Entry:
        w4g128_status_string = staticmethod(strings)

        def __getattr__(self, name):
            return lambda *a: called.append(name) or 0

    monkeypatch.setattr(w, "lib", Entry)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    ws = [gpu(64, dtype="uint8", index=i) for i in (0, 1)]
    on_cpu = torch.zeros(64, dtype=torch.uint8)
    calls = [lambda args, ws: w.w4g128_attend(args, ws, stream=0), lambda args, ws: w.AttendStep(args, ws, stream=0).run(),
             lambda args, ws: w.w4g128_moe(args, ws, stream=0), lambda args, ws: w.MoEStep(args, ws, stream=0).run(),
             lambda args, ws: w.w4g128_sample(args, stream=0), lambda args, ws: w.SampleStep(args, stream=0).run()]
    there = {t: gpu(*s, dtype="bfloat16", index=1) for t, s in (("x", (2, 256)), ("q", (4, 8, 64)), ("logits", (4, 100)))}
    raw = [attend_args(q=there["q"])] * 2 + [moe_args(x=there["x"])] * 2 + [sample_args(logits=there["logits"])] * 2
    for call, good, bad in zip(calls, raw, elsewhere):
        call(good, ws[1])
        assert len(called) == 1
        wrong = [(bad, ws[1])]
        if good is not raw[-1]:  # (sampling has no workspace)
            wrong += [(good, ws[0]), (good, on_cpu)]
        for args, space in wrong:
            with pytest.raises(w.W4G128Error):
                call(args, space)
        assert len(called) == 1
        called.clear()


def test_structs_copied_from_bytes_are_taken():
    """ctypes makes them without the constructor, from raw pointers."""
    for args, call in ((sample_args(vocab=0), lambda a: w.w4g128_sample(a, stream=0)),
                       (attend_args(head_dim=96), lambda a: w.w4g128_attend(a, FAKE, 1 << 40, stream=0)),
                       (moe_args(D=192), lambda a: w.w4g128_moe(a, FAKE, 1 << 40, stream=0))):
        with pytest.raises(w.W4G128Error) as ei:
            call(type(args).from_buffer_copy(bytes(args)))
        assert ei.value.status == E_SHAPE
