"""Argument checks of the calls around the layer (mq_w4a16_linear,
mq_kv4_append, mq_kv4_attention): every violation is refused with its documented
status before anything is enqueued, so no GPU is needed (pointers are fake)."""
import ctypes
import os
import shutil
import subprocess

import pytest

from dense_sparse_w4a4_amd import ops

OK, NULLP, SHAPE, ALIGN, BLOCK, BUDGET, CSR, WS, HIP, ARG = range(10)
P = ctypes.c_void_p(0x1000)
PMIS = ctypes.c_void_p(0x1008)
PODD = ctypes.c_void_p(0x1001)

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
PKG = os.path.join(ROOT, "dense_sparse_w4a4_amd")
HIPCC = "/opt/rocm/bin/hipcc"


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(ops.LIB_PATH):
        from dense_sparse_w4a4_amd import build
        build.build(verbose=False)
    return ops.lib()


def test_w4a16_linear_validation(L):
    def call(**kw):
        a = dict(x=P, dt=0, M=4, K=512, ldx=512, N=512, qw=P, sw=P, b=64, ns=6, rp=P, ci=P, qr=P, sr=P, y=P, ldy=512,
                 ws=None, wsb=0)
        a.update(kw)
        return L.mq_w4a16_linear(*a.values(), None)
    assert call(dt=2) == ARG and call(dt=-1) == ARG
    assert call(b=48) == BLOCK
    assert call(M=-1) == SHAPE and call(M=1 << 20) == SHAPE
    assert call(N=100) == SHAPE and call(N=0) == SHAPE and call(N=1 << 31) == SHAPE
    assert call(K=100) == SHAPE and call(K=0) == SHAPE
    assert call(ldx=504) == SHAPE and call(ldy=504) == SHAPE
    assert call(ns=65) == BUDGET and call(ns=-1) == BUDGET
    for name in ("x", "qw", "sw", "y", "rp", "ci", "qr", "sr"):
        assert call(**{name: None}) == NULLP, name
        assert call(**{name: PMIS}) == ALIGN, name
    assert call(ldx=516) == ALIGN and call(ldy=516) == ALIGN
    assert call(K=(1 << 18) + 128, ldx=1 << 19) == SHAPE
    assert call(M=0, x=None, y=None, qw=None) == OK
    n = ctypes.c_size_t(7)
    w = L.mq_w4a16_linear_workspace
    assert w(4, 512, 512, None) == NULLP
    assert w(4, 500, 512, ctypes.byref(n)) == SHAPE and w(4, 512, 500, ctypes.byref(n)) == SHAPE
    assert w(-1, 512, 512, ctypes.byref(n)) == SHAPE
    for M in (0, 1, 16):
        assert w(M, 512, 8192, ctypes.byref(n)) == OK and n.value == 0
    assert w(50, 5120, 25600, ctypes.byref(n)) == OK and n.value == 3 * 50 * 5120 * 4  # 80 tiles: three splits
    big = dict(M=50, N=5120, K=25600, ldx=25600, ldy=5120, ns=0)
    assert call(**big) == WS
    assert call(**big, ws=P, wsb=3 * 50 * 5120 * 4 - 1) == WS
    assert call(**big, ws=PMIS, wsb=1 << 30) == ALIGN


def test_kv4_append_validation(L):
    def call(**kw):
        a = dict(q=P, ldq=512, k=P, ldk=128, v=P, ldv=128, dt=0, T=3, hq=4, hk=1, D=128, slots=P, pos=P, cs=P, np=9,
                 rot=128, inter=0, wq=P, wk=P, eps=1e-6, kq=P, ksz=P, vq=P, vsz=P, pages=5, page=32, qo=P, ldqo=512,
                 ko=None, vo=None)
        a.update(kw)
        return L.mq_kv4_append(*a.values(), None)
    assert call(dt=3) == ARG
    assert call(D=96) == SHAPE and call(D=256) == SHAPE
    assert call(hq=0) == SHAPE and call(hk=0) == SHAPE and call(hk=3) == SHAPE and call(hk=-1) == SHAPE
    assert call(page=16) == SHAPE and call(page=48) == SHAPE and call(page=1 << 17) == SHAPE
    assert call(pages=0) == SHAPE and call(pages=1 << 31) == SHAPE
    assert call(T=-1) == SHAPE and call(T=1 << 29) == SHAPE
    assert call(ldq=504) == SHAPE and call(ldk=120) == SHAPE and call(ldv=120) == SHAPE and call(ldqo=504) == SHAPE
    assert call(rot=24) == SHAPE and call(rot=144) == SHAPE and call(rot=-16) == SHAPE
    assert call(np=0) == SHAPE
    assert call(eps=-1.0) == ARG and call(eps=float("nan")) == ARG and call(eps=float("inf")) == ARG
    for name in ("q", "k", "v", "slots", "pos", "cs", "wq", "wk", "kq", "ksz", "vq", "vsz", "qo"):
        assert call(**{name: None}) == NULLP, name
    for name in ("q", "k", "v", "cs", "wq", "wk", "kq", "ksz", "vq", "vsz", "qo", "ko", "vo"):
        assert call(**{name: PMIS}) == ALIGN, name
    assert call(slots=ctypes.c_void_p(0x1004)) == ALIGN and call(pos=PODD) == ALIGN
    for name in ("ldq", "ldk", "ldv", "ldqo"):
        assert call(**{name: 516}) == ALIGN, name
    assert call(T=0, q=None, k=None, slots=None) == OK


def test_kv4_attention_validation(L):
    n = ctypes.c_size_t(7)
    w = L.mq_kv4_attention_workspace
    assert w(3, 3, 8, 2, 128, 1, None) == NULLP
    assert w(0, 0, 8, 2, 128, 1, ctypes.byref(n)) == OK and n.value == 0
    assert w(3, 3, 8, 2, 96, 1, ctypes.byref(n)) == SHAPE
    assert w(3, 3, 8, 3, 128, 1, ctypes.byref(n)) == SHAPE
    assert w(3, -1, 8, 2, 128, 1, ctypes.byref(n)) == SHAPE
    assert w(3, 1 << 24, 8, 2, 128, 1, ctypes.byref(n)) == SHAPE
    assert w(3, 3, 8, 2, 128, 0, ctypes.byref(n)) == SHAPE
    assert w(3, 3, 8, 2, 128, 1, ctypes.byref(n)) == OK
    need = n.value

    def call(**kw):
        a = dict(q=P, ldq=1024, dt=0, T=3, hq=8, hk=2, D=128, kq=P, ksz=P, vq=P, vsz=P, pages=5, page=32, bt=P, ldt=4,
                 mp=4, ns=3, kl=P, cu=None, mq=1, causal=1, window=0, scale=0.1, out=P, ldo=1024, lse=None, ws=P,
                 wsb=max(need, 1))
        a.update(kw)
        return L.mq_kv4_attention(*a.values(), None)
    assert call(dt=9) == ARG
    assert call(D=80) == SHAPE and call(hq=7) == SHAPE and call(hk=0) == SHAPE
    assert call(page=33) == SHAPE and call(pages=0) == SHAPE
    assert call(ns=2) == SHAPE and call(T=-1) == SHAPE and call(mq=0) == SHAPE
    assert call(ldq=1016) == SHAPE and call(ldo=1016) == SHAPE
    assert call(mp=5) == SHAPE and call(mp=-1) == SHAPE and call(mp=1 << 26, ldt=1 << 26) == SHAPE
    assert call(window=-1) == ARG
    assert call(scale=float("nan")) == ARG and call(scale=float("-inf")) == ARG
    for name in ("q", "kq", "ksz", "vq", "vsz", "bt", "kl", "out"):
        assert call(**{name: None}) == NULLP, name
    for name in ("q", "kq", "ksz", "vq", "vsz", "out", "ws"):
        assert call(**{name: PMIS}) == ALIGN, name
    for name in ("bt", "kl", "cu", "lse"):
        assert call(**{name: PODD}) == ALIGN, name
    assert call(ldq=1028) == ALIGN and call(ldo=1028) == ALIGN
    if need:
        assert call(ws=None) == WS and call(wsb=need - 1) == WS
    assert call(T=0, ns=0, q=None, out=None, bt=None, kl=None) == OK


def test_kv4_attention_token_counts_leave_room_in_32_bits(L):
    """Positions are 32-bit, and steps are looked at past a sequence's end: the
    most tokens of a table stop 2^16 short of 2^31 (window = -1, checked later,
    stands for a call that is refused for nothing else)."""
    def call(pages, page):
        return L.mq_kv4_attention(P, 1024, 0, 3, 8, 2, 128, P, P, P, P, 5, page, P, 1 << 40, pages, 3, P, None, 1, 1, -1,
                                  0.1, P, 1024, None, P, 1 << 30, None)
    most = (1 << 31) - (1 << 16)
    for page in (32, 64, 4096, 65536):
        assert call(most // page, page) == ARG
        assert call(most // page + 1, page) == SHAPE and call((1 << 31) // page - 1, page) == (
            SHAPE if page < 65536 else ARG)


def test_calls_larger_than_a_launch_are_refused(L):
    """More threads than a launch holds (2^32): refused, not cut short.  ARG: a
    later check, for a call that is refused for nothing else."""
    def append(T, hq, hk, D):
        return L.mq_kv4_append(P, 1 << 40, P, 1 << 40, P, 1 << 40, 0, T, hq, hk, D, P, None, None, 0, 0, 0, None, None,
                               -1.0, P, P, P, P, 5, 32, P, 1 << 40, None, None, None)
    assert append((1 << 26) - 4, 6, 1, 128) == ARG and append((1 << 26) - 3, 6, 1, 128) == SHAPE
    assert append((1 << 27) - 8, 6, 1, 64) == ARG and append((1 << 27) - 7, 6, 1, 64) == SHAPE

    n = ctypes.c_size_t(0)

    def attend(T, seqs, hq, hk, max_q):
        w = L.mq_kv4_attention_workspace(T, seqs, hq, hk, 128, max_q, ctypes.byref(n))
        c = L.mq_kv4_attention(P, 1 << 40, 0, T, hq, hk, 128, P, P, P, P, 5, 32, P, 8, 8, seqs, P, P, max_q, 1, -1, 0.1,
                               P, 1 << 40, None, P, 1 << 62, None)
        assert (w == OK) == (c == ARG) and w in (OK, SHAPE) and c in (ARG, SHAPE)
        return w
    # many sequences, few of them with queries: only those take workgroups
    assert attend(4, (1 << 24) - 1, 4096, 4096, 128) == OK
    assert attend(1 << 20, 1 << 20, 8, 8, 128) == OK
    assert attend(1 << 21, 1 << 21, 8, 8, 128) == SHAPE
    assert attend(1 << 21, 1 << 21, 8, 8, 1) == OK  # the decoding kernel's grid is fixed


@pytest.mark.skipif(not (os.path.exists(HIPCC) and shutil.which("g++")), reason="needs hipcc and g++")
def test_decode_calls_under_host_sanitizers(tmp_path):
    """The host code of these calls with extreme sizes under AddressSanitizer
    and UndefinedBehaviorSanitizer (host code only)."""
    from dense_sparse_w4a4_amd import build
    objdir = os.path.join(PKG, "_build")
    others = [os.path.join(objdir, os.path.basename(s)[:-4] + ".o") for s in build.sources()
              if not s.endswith("api.hip")]
    if not all(os.path.exists(o) for o in others):
        build.build(verbose=False)
    api_o = tmp_path / "api_sanitized.o"
    subprocess.run([HIPCC, *build.FLAGS, "-Xarch_host", "-fsanitize=address", "-Xarch_host",
                    "-fsanitize=undefined", "-Xarch_host", "-fno-sanitize-recover=all",
                    "-fno-omit-frame-pointer", "-c", os.path.join(PKG, "csrc", "api.hip"), "-o", str(api_o)],
                   check=True, capture_output=True)
    exe = tmp_path / "abi_sanitize_decode"
    subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                    f"-I{os.path.join(ROOT, 'include')}", os.path.join(HERE, "csrc", "abi_sanitize_decode.cpp"),
                    str(api_o), *others, "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib",
                    "-o", str(exe)], check=True, capture_output=True)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300, env=env)
    assert out.returncode == 0, out.stdout[-3000:] + out.stderr[-3000:]
    assert "failures 0" in out.stdout
