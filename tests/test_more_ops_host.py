"""Host-side checks of w4g128_append, w4g128_attend8 and w4g128_penalize that
need no GPU: argument structs and refusals, returned before anything is launched."""
import ctypes
import re

import pytest

import int4_weight_only_g128_gb300 as w
from test_ops_host import E_ALIGN, E_CUDA, E_DEVICE, E_INVALID, E_SHAPE, E_WS, FAKE, gpu, header, view


def call(entry, args, ws=FAKE, ws_bytes=1 << 40):
    fn = getattr(w.lib(), entry)
    return fn(ctypes.byref(args), None) if entry == "w4g128_penalize" else fn(ctypes.byref(args), ws, ws_bytes, None)


APPEND = dict(q=FAKE, q_out=FAKE + 0x1000, k_new=FAKE, v_new=FAKE, k_cache=FAKE, v_cache=FAKE, k_scale=FAKE, v_scale=FAKE,
              freqs=FAKE, page_table=FAKE, row_offsets=FAKE, lens=FAKE, q_row=512, q_out_row=512, kv_row=128,
              page_stride=2048, slot_stride=128, head_stride=64, scale_page=2, scale_head=1, table_row=8, rows=4, count=1,
              q_heads=8, kv_heads=2, head_dim=64, rot_dim=64, interleaved=0, pages=8, page_size=16, block=16, max_len=100,
              max_new=4)
ATTEND8 = dict(q=FAKE, k_cache=FAKE, v_cache=FAKE, k_scale=FAKE, v_scale=FAKE, page_table=FAKE, row_offsets=FAKE, lens=FAKE,
               out=FAKE, q_row=512, out_row=512, page_stride=2048, slot_stride=128, head_stride=64, scale_page=2,
               scale_head=1, table_row=8, rows=4, count=1, q_heads=8, kv_heads=2, head_dim=64, pages=8, page_size=16,
               block=16, max_len=100, max_new=4, window=0, sinks=0, scale=0.125)
PENALIZE = dict(logits=FAKE, out=FAKE, history=FAKE, history_start=FAKE, history_len=FAKE, prompt_len=FAKE, repetition=FAKE,
                presence=FAKE, frequency=FAKE, bias_tokens=FAKE, bias_values=FAKE, bias_offsets=FAKE, mask=FAKE,
                row_stride=100, out_stride=100, mask_row=4, history_size=10, bias_size=10, rows=1, vocab=100)


def append(ws=FAKE, ws_bytes=1 << 40, **kw):
    return call("w4g128_append", w.AppendArgs(**{**APPEND, **kw}), ws, ws_bytes)


def attend8(ws=FAKE, ws_bytes=1 << 40, **kw):
    return call("w4g128_attend8", w.Attend8Args(**{**ATTEND8, **kw}), ws, ws_bytes)


def penalize(**kw):
    return call("w4g128_penalize", w.PenalizeArgs(**{**PENALIZE, **kw}))


def test_structs_match_the_header():
    for cls, name in ((w.AppendArgs, "w4g128_append_args"), (w.Attend8Args, "w4g128_attend8_args"),
                      (w.PenalizeArgs, "w4g128_penalize_args")):
        body = re.search(r"typedef struct \{([^}]*)\} " + name + ";", header()).group(1)
        body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
        fields = [f.split()[-1].lstrip("*") for line in body.split(";") if line.strip()
                  for f in line.replace(",", " ,").split(",")]
        assert fields == [f[0] for f in cls._fields_], name


def test_append_refusals():
    assert w.lib().w4g128_append(None, FAKE, 1 << 40, None) == E_INVALID
    for f in ("q", "q_out", "k_new", "v_new", "k_cache", "v_cache", "k_scale", "v_scale", "freqs", "page_table",
              "row_offsets", "lens"):
        assert append(**{f: None}) == E_INVALID, f
    assert append(ws=None) == E_INVALID
    for kw in (dict(rows=0), dict(rows=(1 << 20) + 1), dict(count=0), dict(count=w.MAX_SEQUENCES + 1), dict(max_new=0),
               dict(max_new=(1 << 20) + 1), dict(interleaved=2), dict(interleaved=-1), dict(block=0), dict(rot_dim=0),
               dict(q_heads=0), dict(q=None, q_out=None), dict(q_out=FAKE, q_out_row=520)):
        assert append(**kw) == E_INVALID, kw
    for kw in (dict(q_heads=4097, q_row=1 << 19, q_out_row=1 << 19), dict(q_heads=-1), dict(kv_heads=0), dict(kv_heads=257, kv_row=1 << 15),
               dict(head_dim=96), dict(head_dim=32), dict(rot_dim=80), dict(rot_dim=24), dict(rot_dim=-16), dict(pages=0),
               dict(page_size=8), dict(page_size=24), dict(max_len=0), dict(max_len=(1 << 24) + 1), dict(max_len=129),
               dict(block=3), dict(block=-16), dict(block=32), dict(block=128, page_size=128), dict(q_row=504),
               dict(q_out_row=504), dict(kv_row=120), dict(slot_stride=48), dict(head_stride=48), dict(page_stride=32),
               dict(block=4, scale_page=3, scale_head=4), dict(block=4, scale_page=8, scale_head=3)):
        assert append(**kw) == E_SHAPE, kw
    for f in ("q", "q_out", "k_new", "v_new", "k_cache", "v_cache"):
        assert append(**{f: FAKE + 8}) == E_ALIGN, f
    for f in ("k_scale", "v_scale", "page_table", "row_offsets", "lens"):
        assert append(**{f: FAKE + 2}) == E_ALIGN, f
    assert append(freqs=FAKE + 4) == E_ALIGN
    for f, v in (("q_row", 516), ("q_out_row", 516), ("kv_row", 132), ("page_stride", 2056), ("slot_stride", 136),
                 ("head_stride", 72)):
        assert append(**{f: v}) == E_ALIGN, f
    bf16 = dict(block=0, k_scale=None, v_scale=None, scale_page=0, scale_head=0)
    assert w.w4g128_append_workspace_bytes(w.AppendArgs(**{**APPEND, **bf16, "page_stride": 2056})) > 0  # 8 elements are 16 bytes
    assert append(page_stride=2052, **bf16) == E_ALIGN
    assert append(ws=FAKE + 8) == E_ALIGN
    need = w.w4g128_append_workspace_bytes(w.AppendArgs(**APPEND))
    assert need > 0 and append(ws_bytes=need - 1) == E_WS
    assert w.w4g128_append_workspace_bytes(w.AppendArgs(**{**APPEND, "max_new": 0})) == 0


def test_attend8_refusals():
    assert w.lib().w4g128_attend8(None, FAKE, 1 << 40, None) == E_INVALID
    for f in ("q", "k_cache", "v_cache", "k_scale", "v_scale", "page_table", "row_offsets", "lens", "out"):
        assert attend8(**{f: None}) == E_INVALID, f
    assert attend8(ws=None) == E_INVALID
    for kw in (dict(rows=0), dict(rows=(1 << 20) + 1), dict(count=0), dict(count=w.MAX_SEQUENCES + 1), dict(max_new=0),
               dict(max_new=17), dict(window=-1), dict(sinks=-1, window=5), dict(sinks=4), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(scale=16385.0), dict(scale=-16385.0)):
        assert attend8(**kw) == E_INVALID, kw
    for kw in (dict(q_heads=7), dict(q_heads=34, q_row=4096, out_row=4096), dict(kv_heads=0), dict(head_dim=96),
               dict(head_dim=32), dict(pages=0), dict(page_size=8), dict(page_size=24), dict(max_len=0),
               dict(max_len=(1 << 24) + 1), dict(max_len=129), dict(block=0), dict(block=3), dict(block=-1), dict(block=32),
               dict(block=128, page_size=128), dict(q_row=504), dict(out_row=504), dict(slot_stride=48),
               dict(head_stride=48), dict(page_stride=32), dict(block=4, scale_page=3, scale_head=4),
               dict(block=4, scale_page=8, scale_head=3)):
        assert attend8(**kw) == E_SHAPE, kw
    for f in ("q", "k_cache", "v_cache", "out"):
        assert attend8(**{f: FAKE + 8}) == E_ALIGN, f
    for f in ("k_scale", "v_scale", "page_table", "row_offsets", "lens"):
        assert attend8(**{f: FAKE + 2}) == E_ALIGN, f
    for f, v in (("q_row", 516), ("out_row", 516), ("page_stride", 2056), ("slot_stride", 136), ("head_stride", 72)):
        assert attend8(**{f: v}) == E_ALIGN, f
    assert attend8(ws=FAKE + 8) == E_ALIGN
    need = w.w4g128_attend8_workspace_bytes(w.Attend8Args(**ATTEND8))
    assert need > 0 and attend8(ws_bytes=need - 1) == E_WS
    assert w.w4g128_attend8_workspace_bytes(w.Attend8Args(**{**ATTEND8, "max_new": 0})) == 0
    big = dict(max_len=1 << 24, max_new=16, table_row=1 << 20, q_heads=16, q_row=4096, out_row=4096, kv_heads=1, head_dim=256,
               slot_stride=256, head_stride=256, page_stride=4096)
    assert 0 < w.w4g128_attend8_workspace_bytes(w.Attend8Args(**{**ATTEND8, **big})) < 1 << 30
    # the sums' place does not follow the longest length: a long table costs no more than the call needs
    more = w.w4g128_attend8_workspace_bytes(w.Attend8Args(**{**ATTEND8, **big, "count": 1024}))
    assert 0 < more < 1 << 34


def test_penalize_refusals():
    assert w.lib().w4g128_penalize(None, None) == E_INVALID
    for f in ("logits", "out"):
        assert penalize(**{f: None}) == E_INVALID, f
    for f in ("history_len", "bias_values", "bias_offsets"):
        assert penalize(**{f: None}) == E_INVALID, f
    for kw in (dict(rows=0), dict(rows=w.MAX_SAMPLE_ROWS + 1), dict(history_size=-1), dict(bias_size=-1),
               dict(out_stride=101)):
        assert penalize(**kw) == E_INVALID, kw
    for kw in (dict(vocab=0), dict(vocab=w.MAX_VOCAB + 1, row_stride=1 << 20, out_stride=1 << 20, mask_row=1 << 20),
               dict(row_stride=99, out=FAKE + 64), dict(out_stride=99, out=FAKE + 64), dict(mask_row=3), dict(mask_row=-4)):
        assert penalize(**kw) == E_SHAPE, kw
    assert penalize(logits=FAKE + 1) == E_ALIGN and penalize(out=FAKE + 1) == E_ALIGN
    assert penalize(history_start=FAKE + 4) == E_ALIGN
    for f in ("history", "history_len", "prompt_len", "repetition", "presence", "frequency", "bias_tokens", "bias_values",
              "bias_offsets", "mask"):
        assert penalize(**{f: FAKE + 2}) == E_ALIGN, f


_FAULT_CHILD = """
import sys
sys.path[:0] = [{root!r}, {root!r} + "/tests"]
import test_more_ops_host as t
print(t.append(), t.attend8(), t.penalize(), t.penalize(rows=0))
"""


@pytest.mark.parametrize("mode,status", [("launch", E_CUDA), ("workspace", E_WS)])
def test_host_fault_hook(mode, status):
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "-c", _FAULT_CHILD.format(root=root)], capture_output=True, text=True,
                         env=dict(os.environ, W4G128_FAULT=mode), timeout=120)
    assert out.returncode == 0, out.stderr
    assert [int(v) for v in out.stdout.split()] == [status] * 3 + [E_INVALID]


def test_no_device_is_reported():
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert append() == E_DEVICE and attend8() == E_DEVICE and penalize() == E_DEVICE


def append_tensors(**kw):
    bf = lambda *s: gpu(*s, dtype="bfloat16")  # noqa: E731
    a = {**APPEND, **dict(q=bf(4, 8, 64), q_out=bf(4, 8, 64), k_new=bf(4, 2, 64), v_new=bf(4, 2, 64),
                          k_cache=gpu(8, 16, 2, 64, dtype="uint8"), v_cache=gpu(8, 16, 2, 64, dtype="uint8"),
                          k_scale=gpu(8, 2, 1), v_scale=gpu(8, 2, 1), freqs=gpu(32, dtype="float64"),
                          page_table=gpu(1, 8, dtype="int32"), row_offsets=gpu(2, dtype="int32"), lens=gpu(1, dtype="int32"))}
    return w.AppendArgs(**{**a, **kw})


def attend8_tensors(**kw):
    a = {**ATTEND8, **dict(q=gpu(4, 8, 64, dtype="bfloat16"), out=gpu(4, 8, 64, dtype="bfloat16"),
                           k_cache=gpu(8, 16, 2, 64, dtype="uint8"), v_cache=gpu(8, 16, 2, 64, dtype="uint8"),
                           k_scale=gpu(8, 2, 1), v_scale=gpu(8, 2, 1), page_table=gpu(1, 8, dtype="int32"),
                           row_offsets=gpu(2, dtype="int32"), lens=gpu(1, dtype="int32"))}
    return w.Attend8Args(**{**a, **kw})


def penalize_tensors(**kw):
    i, f = (lambda n: gpu(n, dtype="int32")), gpu
    a = {**PENALIZE, **dict(logits=gpu(2, 100, dtype="bfloat16"), out=gpu(2, 100, dtype="bfloat16"), history=i(10),
                            history_start=gpu(2, dtype="int64"), history_len=i(2), prompt_len=i(2), repetition=f(2),
                            presence=f(2), frequency=f(2), bias_tokens=i(10), bias_values=f(10), bias_offsets=i(3),
                            mask=gpu(2, 4, dtype="int32"), rows=2)}
    return w.PenalizeArgs(**{**a, **kw})


def test_tensors_are_checked_by_the_binding():
    """Element sizes, reach and layout of every tensor; one device."""
    pytest.importorskip("torch")
    append_tensors(), attend8_tensors(), penalize_tensors()  # as they should be
    bf16 = dict(block=0, k_scale=None, v_scale=None, k_cache=gpu(8, 16, 2, 64, dtype="bfloat16"),
                v_cache=gpu(8, 16, 2, 64, dtype="bfloat16"))
    append_tensors(**bf16)
    append_tensors(q=view(gpu(4, 600, dtype="bfloat16"), lambda t: t[:, :512]), q_row=600)
    attend8_tensors(k_cache=view(gpu(8, 2, 16, 64, dtype="uint8"), lambda t: t.transpose(1, 2)), slot_stride=64,
                    head_stride=1024)
    penalize_tensors(mask=gpu(1, 4, dtype="int32"), mask_row=0)
    wrong = [(append_tensors, dict(bf16, k_cache=gpu(8, 16, 2, 64, dtype="uint8"))),
             (append_tensors, dict(k_cache=gpu(8, 16, 2, 64, dtype="bfloat16"))),
             (append_tensors, dict(freqs=gpu(32))), (append_tensors, dict(freqs=gpu(31, dtype="float64"))),
             (append_tensors, dict(k_scale=gpu(8, 2, 1, dtype="float64"))), (append_tensors, dict(v_scale=gpu(7, 2, 1))),
             (append_tensors, dict(k_cache=gpu(7, 16, 2, 64, dtype="uint8"))), (append_tensors, dict(q=gpu(3, 8, 64, dtype="bfloat16"))),
             (append_tensors, dict(k_new=gpu(3, 2, 64, dtype="bfloat16"))), (append_tensors, dict(page_table=gpu(1, 6, dtype="int32"))),
             (append_tensors, dict(lens=gpu(1, dtype="int64"))), (append_tensors, dict(row_offsets=gpu(1, dtype="int32"))),
             (append_tensors, dict(lens=gpu(1, dtype="int32", index=1))),
             (attend8_tensors, dict(v_cache=gpu(8, 16, 2, 64, dtype="bfloat16"))),
             (attend8_tensors, dict(k_scale=gpu(8, 2, 1, dtype="bfloat16"))), (attend8_tensors, dict(v_scale=gpu(7, 2, 1))),
             (attend8_tensors, dict(out=gpu(3, 8, 64, dtype="bfloat16"))),
             (attend8_tensors, dict(k_cache=view(gpu(8, 16, 64, 2, dtype="uint8"), lambda t: t.transpose(2, 3)))),
             (penalize_tensors, dict(history_start=gpu(2, dtype="int32"))), (penalize_tensors, dict(out=gpu(2, 100))),
             (penalize_tensors, dict(bias_offsets=gpu(2, dtype="int32"))), (penalize_tensors, dict(history=gpu(9, dtype="int32"))),
             (penalize_tensors, dict(bias_values=gpu(9))), (penalize_tensors, dict(mask=gpu(2, 3, dtype="int32"))),
             (penalize_tensors, dict(frequency=view(gpu(2, 2), lambda t: t[:, 0]))),
             (penalize_tensors, dict(logits=view(gpu(100, 2, dtype="bfloat16"), lambda t: t.t())))]
    for make, bad in wrong:
        with pytest.raises(w.W4G128Error) as ei:
            make(**bad)
        assert ei.value.status == E_INVALID, bad


def test_calls_on_another_device_are_refused(monkeypatch):
    torch = pytest.importorskip("torch")
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    ws = gpu(256, dtype="uint8")
    for fn in (lambda: w.w4g128_append(append_tensors(), ws, stream=0), lambda: w.AppendStep(append_tensors(), ws, stream=0),
               lambda: w.w4g128_attend8(attend8_tensors(), ws, stream=0), lambda: w.Attend8Step(attend8_tensors(), ws, stream=0),
               lambda: w.w4g128_penalize(penalize_tensors(), stream=0), lambda: w.PenalizeStep(penalize_tensors(), stream=0),
               lambda: w.w4g128_append(w.AppendArgs(**APPEND), ws, stream=0),
               lambda: w.w4g128_attend8(w.Attend8Args(**ATTEND8), ws, stream=0)):
        with pytest.raises(w.W4G128Error) as ei:
            fn()
        assert ei.value.status == E_INVALID


def test_structs_copied_from_bytes_are_taken():
    for args, fn in ((w.AppendArgs(**{**APPEND, "head_dim": 96}), lambda a: w.w4g128_append(a, FAKE, 1 << 40, stream=0)),
                     (w.Attend8Args(**{**ATTEND8, "head_dim": 96}), lambda a: w.w4g128_attend8(a, FAKE, 1 << 40, stream=0)),
                     (w.PenalizeArgs(**{**PENALIZE, "vocab": 0}), lambda a: w.w4g128_penalize(a, stream=0))):
        with pytest.raises(w.W4G128Error) as ei:
            fn(type(args).from_buffer_copy(bytes(args)))
        assert ei.value.status == E_SHAPE
