"""What the host API asks of CUDA, and what it does when a launch fails: csrc/pv_api.cu and
csrc/pv_plan.cu are built with tests/fake_cuda.cpp in place of the runtime and the kernels, which
writes each call to a log.  No device is needed."""
import ctypes
import os
import shutil
import subprocess
import sys

import pytest

from same_step_kv_b200 import pv

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
KV, WS, MEANS = 1 << 40, 1 << 41, 1 << 42      # addresses that nothing reads
F0 = 3


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    gxx = shutil.which("g++")
    assert gxx, "g++ is not available"
    so = str(tmp_path_factory.mktemp("host") / "libpv_host.so")
    src = [os.path.join(ROOT, "same_step_kv_b200", "csrc", f) for f in ("pv_api.cu", "pv_plan.cu")]
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    subprocess.run([gxx, "-std=c++17", "-O1", "-fPIC", "-shared", "-fvisibility=hidden", "-Wl,-Bsymbolic",
                    "-Wl,--no-undefined", "-I", cuda, "-x", "c++", *src,
                    os.path.join(ROOT, "tests", "fake_cuda.cpp"), "-o", so, "-lpthread"],
                   check=True, capture_output=True, text=True)
    m = ctypes.CDLL(so)
    for name, (args, res) in pv._SIGS.items():
        if f := getattr(m, name, None):          # (pv_noalloc.cu is not built here)
            f.argtypes, f.restype = args, res
    m.fake_log.restype = ctypes.c_char_p
    m.so = so
    return m


def log(lib):
    return lib.fake_log().decode().split("\n")[:-1]


def moves(lib):
    n = lib.fake_moves(None, 0)
    a = (ctypes.c_int * max(n, 1))()
    lib.fake_moves(a, n)
    return list(zip(a[0:n:2], a[1:n:2]))


class Store:
    def __init__(self, lib, cfg, pages=None):
        self.lib, self.cfg, self.h = lib, cfg, ctypes.c_void_p()
        lib.fake_reset(-1)
        big = 1 << 62
        args = (KV, big, WS, big)
        assert (lib.pv_kv_init(ctypes.byref(self.h), ctypes.byref(cfg), *args) if pages is None else
                lib.pv_kv_init_paged(ctypes.byref(self.h), ctypes.byref(cfg), pages, *args)) == pv.PV_OK

    def set(self, stream, chunk, phase=pv.PV_PHASE_STEADY):
        st = pv.pv_kv_state()
        st.phase, st.chunk = phase, chunk
        assert self.lib.pv_kv_set_state(self.h, stream, ctypes.byref(st)) == pv.PV_OK

    def state(self, stream):
        st = pv.pv_kv_state()
        assert self.lib.pv_kv_get_state(self.h, stream, ctypes.byref(st)) == pv.PV_OK
        return st.phase, st.chunk, st.fill, st.slot, list(st.slot_frame)

    def pages(self, stream):
        sink, ring = ctypes.c_int(), (ctypes.c_int * pv.PV_MAX_RING)()
        assert self.lib.pv_kv_page_table(self.h, stream, ctypes.byref(sink), ring) == pv.PV_OK
        return sink.value, list(ring)[:self.cfg.ring_slots]

    def free(self):
        a, b = ctypes.c_int(), ctypes.c_int()
        assert self.lib.pv_kv_free_pages(self.h, ctypes.byref(a), ctypes.byref(b)) == pv.PV_OK
        return a.value, b.value


def of_many_pages(lib):
    """17 streams of 67 one-token pages, the second one ended: 1,005 pages to move."""
    s = Store(lib, pv.make_config(1, 1, 64, 1, 1, first_frames=F0, ring_slots=64, steps=1, max_streams=17,
                                  max_frames=256), 17 * 67)
    for i in range(17):
        s.set(i, 64)
    assert lib.pv_kv_release(s.h, 1) == pv.PV_OK
    return s


def run_of_67(first):
    return first, list(range(first + F0, first + 67))


def test_compaction_in_several_launches(lib):
    s = of_many_pages(lib)
    lib.fake_reset(-1)
    n = ctypes.c_int()
    assert lib.pv_kv_compact(s.h, ctypes.byref(n), None) == pv.PV_OK
    assert n.value == 15 * 67 and log(lib) == ["launch copy"] * 3
    assert moves(lib) == [(134 + i, 67 + i) for i in range(15 * 67)]
    assert s.pages(0) == run_of_67(0)
    assert [s.pages(i) for i in range(2, 17)] == [run_of_67((i - 1) * 67) for i in range(2, 17)]
    lib.pv_kv_destroy(s.h)


def test_compaction_whose_first_launch_fails_changes_nothing(lib):
    s = of_many_pages(lib)
    before = [(s.pages(i), s.state(i)) for i in range(17)], s.free()
    lib.fake_reset(0)
    n = ctypes.c_int(5)
    assert lib.pv_kv_compact(s.h, ctypes.byref(n), None) == pv.PV_ERR_CUDA
    assert n.value == 0 and moves(lib) == []
    assert ([(s.pages(i), s.state(i)) for i in range(17)], s.free()) == before
    lib.fake_reset(-1)
    assert lib.pv_kv_compact(s.h, None, None) == pv.PV_OK
    lib.pv_kv_destroy(s.h)


@pytest.mark.parametrize("k", [1, 2])
def test_compaction_that_fails_half_way_ends_the_streams_that_it_moves(lib, k):
    """Pages have moved and others have not: no stream may read what it held there."""
    s = of_many_pages(lib)
    kept = s.pages(0), s.state(0)
    lib.fake_reset(k)
    n = ctypes.c_int(5)
    assert lib.pv_kv_compact(s.h, ctypes.byref(n), None) == pv.PV_ERR_CUDA
    assert n.value == 0 and len(moves(lib)) == 480 * k
    assert (s.pages(0), s.state(0)) == kept
    for i in range(1, 17):
        assert s.state(i)[:2] == (pv.PV_PHASE_NEW, -1) and s.pages(i) == (-1, [-1] * 64)
    assert s.free() == (16 * 67, 16 * 67)
    lib.fake_reset(-1)
    ids = (ctypes.c_int * 1)(3)
    assert lib.pv_chunk_attn(s.h, 1, ids, 0, 0, 256, 256, None, None) == pv.PV_ERR_STATE
    assert lib.pv_rope_append(s.h, 1, ids, 0, 0, 256, 256, 256, 256, None) == pv.PV_ERR_STATE
    # the store serves new ones
    assert lib.pv_kv_begin_chunk(s.h, 3, F0) == pv.PV_OK
    assert lib.pv_rope_append(s.h, 1, ids, 0, 0, 256, 256, 256, 256, None) == pv.PV_OK
    assert lib.pv_chunk_attn(s.h, 1, ids, 0, 0, 256, 256, None, None) == pv.PV_OK
    assert log(lib) == ["launch rope", "launch block attention"]
    lib.pv_kv_destroy(s.h)


@pytest.mark.parametrize("pages", [None, 20])
def test_fork_whose_copy_fails_changes_nothing(lib, pages):
    s = Store(lib, pv.make_config(1, 2, 64, 4, 4, first_frames=F0, ring_slots=3, steps=2, max_streams=4,
                                  max_frames=64), pages)
    s.set(0, 2)
    free = s.free()
    lib.fake_reset(0)
    dst = (ctypes.c_int * 2)(1, 3)
    assert lib.pv_kv_fork(s.h, 0, 2, dst, 1, None) == pv.PV_ERR_CUDA
    assert s.free() == free and [s.state(i)[0] for i in (1, 2, 3)] == [pv.PV_PHASE_NEW] * 3
    lib.fake_reset(-1)
    assert lib.pv_kv_fork(s.h, 0, 2, dst, 1, None) == pv.PV_OK
    assert log(lib) == ["launch copy"] and s.state(3) == s.state(0)
    lib.pv_kv_destroy(s.h)


# ------------------------------------------------------------------ set-up calls are complete when they return
def waits_after(lines, what):
    """Whether the log holds a wait behind the last line that begins with `what`."""
    last = max(i for i, x in enumerate(lines) if x.startswith(what))
    return any(x.startswith("wait") for x in lines[last + 1:])


@pytest.mark.parametrize("pages", [None, 12])
def test_attached_means_are_clear_when_the_call_returns(lib, pages):
    """Calls on a stream that does not wait for the default one may follow at once."""
    s = Store(lib, pv.make_config(1, 2, 64, 4, 4, first_frames=F0, ring_slots=3, steps=2, max_streams=2,
                                  max_frames=64), pages)
    n = ctypes.c_size_t()
    assert lib.pv_kv_summary_bytes(s.h, ctypes.byref(n)) == pv.PV_OK
    lib.fake_reset(-1)
    assert lib.pv_kv_set_summaries(s.h, MEANS, n.value) == pv.PV_OK
    assert waits_after(log(lib), "memset")
    assert lib.pv_kv_begin_chunk(s.h, 0, F0) == pv.PV_OK
    ids = (ctypes.c_int * 1)(0)
    lib.fake_reset(-1)
    assert lib.pv_block_summarize(s.h, 1, ids, 0, 0, 77) == pv.PV_OK
    assert lib.pv_kv_set_summaries(s.h, None, 0) == pv.PV_OK
    assert log(lib) == ["launch means"]
    lib.pv_kv_destroy(s.h)


@pytest.mark.parametrize("pages", [None, 12])
def test_a_store_is_ready_when_the_call_returns(lib, pages):
    """The zero fill and the RoPE table (copied from pageable memory, which may return before the
    copy has reached the device)."""
    Store(lib, pv.make_config(1, 2, 64, 4, 4, first_frames=F0, ring_slots=3, steps=2, max_streams=2,
                              max_frames=64), pages)
    lines = log(lib)
    assert lines.count("memset") == 2 and "memcpy" in lines
    assert waits_after(lines, "memset") and waits_after(lines, "memcpy")


# ------------------------------------------------------------------ NULL outputs
NULLS = {
    "pv_block_attn_dense_ws_bytes": "lib.pv_block_attn_dense_ws_bytes(5, 300, 2, 64, 2, None)",
    "pv_attn_dense_ws_bytes": "lib.pv_attn_dense_ws_bytes(5, 300, 2, 64, None)",
    "pv_kv_paged_required_bytes": "lib.pv_kv_paged_required_bytes(byref(cfg), 9, None, None)",
    "pv_kv_paged_required_bytes, config": "lib.pv_kv_paged_required_bytes(None, 9, None, None)",
    "pv_kv_init_paged": "lib.pv_kv_init_paged(None, byref(cfg), 9, None, 0, None, 0)",
    "pv_kv_init_paged, config": "lib.pv_kv_init_paged(byref(h), None, 9, None, 0, None, 0)",
    "pv_kv_summary_bytes": "lib.pv_kv_summary_bytes(h, None)",
    "pv_kv_free_pages": "lib.pv_kv_free_pages(h, None, None)",
    "pv_kv_page_table": "lib.pv_kv_page_table(h, 0, None, None)",
    "pv_kv_get_state": "lib.pv_kv_get_state(h, 0, None)",
    "pv_kv_set_state": "lib.pv_kv_set_state(h, 0, None)",
    "pv_kv_row_offset": "lib.pv_kv_row_offset(h, 0, 0, 0, 0, 0, None, None)",
    "pv_kv_fork": "lib.pv_kv_fork(h, 0, 1, None, 0, None)",
    "pv_block_summarize": "lib.pv_block_summarize(dev, 1, None, 0, 0, None)",
    "pv_block_select": "lib.pv_block_select(dev, 1, None, 0, 0, 256, 2, 0, 256, None)",
    "pv_block_select, tensors": "lib.pv_block_select(dev, 1, one, 0, 0, None, 2, 0, None, None)",
    "pv_block_attn": "lib.pv_block_attn(dev, 1, None, 0, 0, 256, 256, 2, 256, None, None)",
    "pv_block_attn, tensors": "lib.pv_block_attn(dev, 1, one, 0, 0, None, 256, 2, None, None, None)",
    "pv_chunk_attn": "lib.pv_chunk_attn(dev, 1, None, 0, 0, 256, 256, None, None)",
}


@pytest.mark.parametrize("name", NULLS)
def test_null_pointers_are_refused(lib, name):
    """In a process of its own: what takes a NULL pointer for granted ends it."""
    code = f"""
import ctypes
from ctypes import byref
from same_step_kv_b200 import pv
lib = ctypes.CDLL({lib.so!r})
for n, (a, r) in pv._SIGS.items():
    if f := getattr(lib, n, None):
        f.argtypes, f.restype = a, r
cfg = pv.make_config(1, 2, 64, 4, 4, first_frames=3, ring_slots=3, steps=2, max_streams=2, max_frames=64)
h, dev = ctypes.c_void_p(), ctypes.c_void_p()
assert lib.pv_kv_init_paged(byref(h), byref(cfg), 9, None, 0, None, 0) == 0
assert lib.pv_kv_init_paged(byref(dev), byref(cfg), 9, {KV}, 1 << 62, {WS}, 1 << 62) == 0
assert lib.pv_kv_set_summaries(dev, {MEANS}, 1 << 62) == 0
one = (ctypes.c_int * 1)(0)
assert lib.pv_kv_begin_chunk(h, 0, 3) == 0 and lib.pv_kv_begin_chunk(dev, 0, 3) == 0
assert {NULLS[name]} == pv.PV_ERR_INVALID_ARG
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, f"{r.returncode} {r.stderr[-500:]}"


def test_a_shared_page_is_written_by_its_last_holder_only(lib):
    """A branch taken with its current page shared: starting the next chunk does not give the page up."""
    s = Store(lib, pv.make_config(1, 2, 64, 4, 4, first_frames=F0, ring_slots=3, steps=2, max_streams=2,
                                  max_frames=64), 12)
    s.set(0, 2)
    one = (ctypes.c_int * 1)(1)
    append = lambda i: lib.pv_rope_append(s.h, 1, (ctypes.c_int * 1)(i), 0, 0, 256, 256, 256, 256, None)  # noqa: E731
    assert append(0) == pv.PV_OK
    assert lib.pv_kv_fork(s.h, 0, 1, one, 0, None) == pv.PV_OK
    assert append(0) == append(1) == pv.PV_ERR_STATE
    assert lib.pv_kv_begin_chunk(s.h, 0, 1) == pv.PV_OK
    assert append(0) == pv.PV_OK and append(1) == pv.PV_ERR_STATE
    assert lib.pv_kv_release(s.h, 0) == pv.PV_OK
    assert append(1) == pv.PV_OK
    lib.pv_kv_destroy(s.h)


def test_a_failed_launch_is_reported_once(lib):
    """The call after it is judged by itself."""
    s = Store(lib, pv.make_config(1, 2, 64, 4, 4, first_frames=F0, ring_slots=3, steps=2, max_streams=2,
                                  max_frames=64), 12)
    s.set(0, 2)
    lib.fake_reset(0)
    dst = (ctypes.c_int * 1)(1)
    assert lib.pv_kv_fork(s.h, 0, 1, dst, 1, None) == pv.PV_ERR_CUDA
    assert lib.pv_chunk_attn(s.h, 1, (ctypes.c_int * 1)(0), 0, 0, 256, 256, None, None) == pv.PV_OK
    assert log(lib) == ["launch block attention"]
    lib.pv_kv_destroy(s.h)


@pytest.mark.parametrize("pages", [None, 12])
def test_buffers_of_another_device_are_refused(lib, pages):
    """Kernels go to the current device: one that reads another's memory would fault."""
    cfg = pv.make_config(1, 2, 64, 4, 4, first_frames=F0, ring_slots=3, steps=2, max_streams=2, max_frames=64)
    far, big = 1 << 50, 1 << 62
    for kv, ws in ((KV + far, WS), (KV, WS + far), (KV + far, WS + far)):
        lib.fake_reset(-1)
        h = ctypes.c_void_p(1)
        st = (lib.pv_kv_init(ctypes.byref(h), ctypes.byref(cfg), kv, big, ws, big) if pages is None else
              lib.pv_kv_init_paged(ctypes.byref(h), ctypes.byref(cfg), pages, kv, big, ws, big))
        assert st == pv.PV_ERR_INVALID_ARG and not h.value and log(lib) == []
    s = Store(lib, cfg, pages)
    lib.fake_reset(-1)
    assert lib.pv_kv_set_summaries(s.h, MEANS + far, big) == pv.PV_ERR_INVALID_ARG and log(lib) == []
    assert lib.pv_kv_begin_chunk(s.h, 0, F0) == pv.PV_OK
    assert lib.pv_block_summarize(s.h, 1, (ctypes.c_int * 1)(0), 0, 0, None) == pv.PV_ERR_STATE
    assert lib.pv_kv_set_summaries(s.h, MEANS, big) == pv.PV_OK
    lib.pv_kv_destroy(s.h)
