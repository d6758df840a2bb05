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
    for name in ("MAX_SAMPLE_ROWS", "MAX_VOCAB"):
        assert re.search(rf"#define W4G128_{name} {getattr(w, name)}\b", text), name


def test_structs_match_the_header():
    """Field names and order of each argument struct."""
    for cls, name in ((w.SampleArgs, "w4g128_sample_args"),):
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
