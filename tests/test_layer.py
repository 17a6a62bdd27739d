"""CPU tests of the calls of a layer over a paged cache: exports, argument checks of the C entry
points and of the Python calls, and the kernels as compiled.  No GPU call is made: accepted
arguments are only tried on a build whose launchers are stand-ins."""
import ctypes
import glob
import os
import re
import shutil
import subprocess

import pytest

torch = pytest.importorskip("torch")

import bmmc_affine_index_amd as bm  # noqa: E402
from bmmc_affine_index_amd import layer as ly  # noqa: E402
from bmmc_affine_index_amd import tokens as tk  # noqa: E402

import matrix_waits  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TESTS = os.path.join(ROOT, "tests")
CSRC = os.path.join(ROOT, "bmmc_affine_index_amd", "csrc", "layer")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
INCLUDE = ["-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I" + os.path.join(ROOT, "include")]
ACCEPTED = bm.ERR_HIP  # what the stand-in launchers return
BAD, ALIAS, OK = bm.ERR_INVALID_ARG, bm.ERR_ALIAS, bm.OK


def test_library_exports_every_header_function():
    header = open(os.path.join(ROOT, "include", "bmmc_layer.h")).read()
    names = set(re.findall(r"^\S[^;()]*?\b(bmmc_\w+)\s*\(", header, flags=re.M))
    assert names == set(ly.LAYER_EXPORTED)
    L = ly.layer_lib()
    for name in names:
        assert hasattr(L, name), name


def test_struct_layouts_match_header(tmp_path):
    structs = {c.__name__: c for c in (ly.bmmc_scaled_cache, ly.bmmc_attention)}
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "bmmc_layer.h"', "int main(void) {"]
    for name, cls in structs.items():
        lines.append('printf("%s %%zu\\n", sizeof(%s));' % (name, name))
        for field, _ in cls._fields_:
            lines.append('printf("%s.%s %%zu\\n", offsetof(%s, %s));' % (name, field, name, field))
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["return 0; }"]))
    subprocess.check_call(["gcc", "-I" + os.path.join(ROOT, "include"), str(src), "-o", str(exe)])
    out = dict(l.split() for l in subprocess.check_output([str(exe)]).decode().splitlines())
    for name, cls in structs.items():
        assert int(out[name]) == ctypes.sizeof(cls), name
        for field, _ in cls._fields_:
            assert int(out[name + "." + field]) == getattr(cls, field).offset, (name, field)


# --------------------------------------------------------------------------
# The kernels as compiled
# --------------------------------------------------------------------------

@pytest.mark.skipif(not os.path.exists(HIPCC), reason="needs hipcc")
@pytest.mark.parametrize("src", [os.path.basename(p) for p in sorted(glob.glob(os.path.join(CSRC, "*.hip")))])
def test_every_kernel_has_a_body_and_its_waits(src, tmp_path):
    """Undefined behaviour can leave a kernel without instructions; and a product's result that is
    read behind a branch has been seen to be read too early."""
    out = tmp_path / (src + ".s")
    subprocess.run([HIPCC, "-O3", "-std=c++17", "-I" + os.path.join(ROOT, "include"),
                    "--offload-arch=gfx950", "-Xclang", "-target-feature", "-Xclang",
                    "-packed-fp32-ops", "-munsafe-fp-atomics", "--cuda-device-only", "-S", "-o", str(out),
                    os.path.join(CSRC, src)], check=True, capture_output=True, timeout=900)
    s = out.read_text()
    kernels = re.findall(r"^\s*\.amdhsa_kernel\s+(\S+)", s, flags=re.M)
    assert kernels
    for name in kernels:
        start = s.index("\n%s:" % name)
        ins = [l.strip() for l in s[start:s.index(".Lfunc_end", start)].splitlines()[1:]]
        assert any(l.startswith("s_endpgm") for l in ins), name
    assert matrix_waits.find(s) == []


def test_early_uses_are_found():
    """The search itself, on lines made by hand."""
    def text(*lines):
        return "\n_Zk:\n" + "\n".join("\t" + l if not l.startswith(".") else l for l in lines) + "\n.Lfunc_end0:\n"
    product = "v_mfma_f32_16x16x32_bf16 a[0:3], v[0:3], v[4:7], a[0:3]"
    read = "v_accvgpr_read_b32 v9, a3"
    assert matrix_waits.find(text(product, read))
    assert matrix_waits.find(text(product, "s_nop 5", read))
    assert not matrix_waits.find(text(product, "s_nop 6", read))
    assert not matrix_waits.find(text(product, "v_accvgpr_read_b32 v9, a4", "s_nop 5", read))
    assert not matrix_waits.find(text(product, product, "s_nop 6", read))
    # behind a branch that is taken, and on the way past it
    assert matrix_waits.find(text(product, "s_cbranch_vccnz .LBB0_2", "s_nop 15", ".LBB0_2:", read))
    assert not matrix_waits.find(text(product, "s_nop 7", "s_cbranch_vccnz .LBB0_2", "s_nop 1", ".LBB0_2:", read))
    # as a factor of another product, or overwritten
    assert matrix_waits.find(text(product, "v_mfma_f32_16x16x32_bf16 a[8:11], a[0:3], v[4:7], a[8:11]"))
    assert matrix_waits.find(text(product, "v_accvgpr_write_b32 a1, v3"))


# --------------------------------------------------------------------------
# The C entry points' checks, on a build whose launchers are stand-ins
# --------------------------------------------------------------------------

@pytest.fixture(scope="module")
def host(tmp_path_factory):
    if shutil.which("g++") is None or not os.path.exists("/opt/rocm/lib"):
        pytest.skip("needs g++ and the ROCm runtime library")
    so = str(tmp_path_factory.mktemp("host") / "liblayer_host.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-fsanitize=undefined",
                    "-fno-sanitize-recover=undefined", *INCLUDE, *sorted(glob.glob(os.path.join(CSRC, "*.cpp"))),
                    os.path.join(TESTS, "layer_stubs.cpp"), "-L/opt/rocm/lib", "-lamdhip64",
                    "-Wl,-rpath,/opt/rocm/lib", "-o", so], check=True, timeout=300)
    L = ctypes.CDLL(so)
    real = ly.layer_lib()
    for name in ly.LAYER_EXPORTED:
        getattr(L, name).argtypes = getattr(real, name).argtypes
        getattr(L, name).restype = getattr(real, name).restype
    return L


A, B, C, D, E, G = (0x100000000 * k for k in range(1, 7))  # addresses nothing is read from


def _cache(data, dim=64, heads=2, page=16, kind=tk.BF16, **changes):
    c = dict(data=data, scale=None, page_stride=page * heads * dim, place_stride=heads * dim,
             head_stride=dim, scale_page=0, scale_place=0, scale_head=0, type=kind)
    c.update(changes)
    return ly.bmmc_scaled_cache(**c)


def _attention(**changes):
    a = dict(q=A, out=B, q_token=8 * 64, q_head=64, out_token=8 * 64, out_head=64, tokens=10, q_heads=8,
             heads=2, table=C, lengths=C + 0x1000, starts=C + 0x2000, pages=100, page_size=16, batch=3,
             table_width=20, table_stride=20, window=0, scale=0.125, k_dim=64, v_dim=64, type=tk.BF16,
             clear_rest=0)
    a.update(changes)
    return ly.bmmc_attention(**a)


@pytest.mark.parametrize("changes,status", [
    ({}, ACCEPTED), ({"tokens": 0}, OK), ({"batch": 0, "table": None, "lengths": None}, ACCEPTED),
    ({"batch": 10, "starts": None}, ACCEPTED), ({"starts": None}, BAD), ({"tokens": -1}, BAD), ({"tokens": 1 << 31}, BAD),
    ({"tokens": (1 << 31) - 1, "q_token": 0, "out_token": 512}, BAD), ({"heads": 3}, BAD), ({"heads": 0}, BAD),
    ({"q_heads": 1}, BAD), ({"q_heads": 1 << 17}, BAD), ({"k_dim": 7}, BAD), ({"k_dim": 513}, BAD), ({"v_dim": 7}, BAD),
    ({"v_dim": 513}, BAD), ({"type": tk.E4M3}, BAD), ({"type": 7}, BAD), ({"window": -1}, BAD), ({"window": 1 << 62}, ACCEPTED),
    ({"scale": 0.0}, BAD), ({"scale": -1.0}, BAD), ({"scale": float("nan")}, BAD), ({"scale": float("inf")}, BAD),
    ({"pages": -1}, BAD), ({"page_size": 0}, BAD), ({"page_size": 1 << 31}, BAD), ({"table": None}, BAD), ({"table": C + 2}, BAD),
    ({"table_width": 0, "table": None}, ACCEPTED), ({"table_width": 1 << 31}, BAD), ({"table_stride": -1}, BAD), ({"lengths": None}, BAD), ({"lengths": C + 2}, BAD),
    ({"starts": C + 2}, BAD), ({"q": None}, BAD), ({"q": A + 1}, BAD), ({"out": None}, BAD), ({"out": B + 1}, BAD),
    ({"q_token": -1}, BAD), ({"out_head": 1 << 41}, BAD), ({"q_token": 0}, ACCEPTED), ({"out_token": 0}, ALIAS),
    ({"out_head": 63}, ALIAS), ({"out": A}, ALIAS), ({"out": A + 10240 - 2}, ALIAS), ({"out": A + 10240}, ACCEPTED),
    ({"out": D + 64}, ALIAS), ({"out": E - 2}, ALIAS), ({"batch": -1}, BAD), ({"batch": 1 << 31}, BAD)])
def test_attention_refusals(host, changes, status):
    a = _attention(**changes)
    if status != OK:
        need = host.bmmc_cache_attention_workspace(a)
        work = 1 << 40
    else:
        need, work = 0, None
    assert host.bmmc_cache_attention(a, _cache(D), _cache(E), work, max(need, 0), None) == status


@pytest.mark.parametrize("k,v,status", [
    (dict(data=D), dict(data=E), ACCEPTED), (dict(data=D), dict(data=D), ACCEPTED), (dict(data=None), dict(data=E), BAD),
    (dict(data=D + 1), dict(data=E), BAD), (dict(data=D, scale=G), dict(data=E), BAD), (dict(data=D, kind=tk.F16), dict(data=E), BAD),
    (dict(data=D, page_stride=-1), dict(data=E), BAD), (dict(data=D, page_stride=0), dict(data=E), ACCEPTED),
    (dict(data=D, kind=tk.E4M3, scale=G), dict(data=E), BAD), (dict(data=D, kind=tk.E4M3), dict(data=E, kind=tk.E4M3, scale=G), BAD),
    (dict(data=D + 1, kind=tk.E4M3, scale=G), dict(data=E, kind=tk.E4M3, scale=G), ACCEPTED),
    (dict(data=D, kind=tk.E4M3, scale=G + 2), dict(data=E, kind=tk.E4M3, scale=G), BAD),
    (dict(data=D, kind=tk.E4M3, scale=G, scale_page=-1), dict(data=E, kind=tk.E4M3, scale=G), BAD),
    (dict(data=D, kind=tk.E4M3, scale=B + 16), dict(data=E, kind=tk.E4M3, scale=G), ALIAS)])
def test_attention_refuses_caches(host, k, v, status):
    a = _attention()
    need = host.bmmc_cache_attention_workspace(a)
    assert host.bmmc_cache_attention(a, _cache(**k), _cache(**v), 1 << 40, need, None) == status


def test_attention_does_not_write_its_indexes(host):
    """The result and the workspace share no byte with the table, the lengths or the starts, which may
    lie between the result's heads."""
    a = _attention()
    need = host.bmmc_cache_attention_workspace(a)
    k, v = _cache(D), _cache(E)
    end = B + 10 * 8 * 64 * 2
    for name, size in (("table", 3 * 20 * 4), ("lengths", 3 * 4), ("starts", 4 * 4)):
        for at, status in ((B, ALIAS), (B - size + 4, ALIAS), (B - size, ACCEPTED), (end - 4, ALIAS), (end, ACCEPTED)):
            assert host.bmmc_cache_attention(_attention(**{name: at}), k, v, 1 << 40, need, None) == status, (name, at)
        for at, status in (((1 << 40) - size, ACCEPTED), ((1 << 40) - size + 4, ALIAS), ((1 << 40) + need - 4, ALIAS),
                           ((1 << 40) + need, ACCEPTED)):
            assert host.bmmc_cache_attention(_attention(**{name: at}), k, v, 1 << 40, need, None) == status, (name, at)
    # 16 bytes of lengths and starts in the 64 that follow each head, and a table's rows
    for name, inside in (("lengths", 12), ("starts", 16)):
        between = dict(out_head=64 + 32, out_token=8 * 96, **{name: B + 96 * 2 * 5 + 128})
        assert host.bmmc_cache_attention(_attention(**between), k, v, 1 << 40, need, None) == ACCEPTED
        between[name] += 64 - inside + 4
        assert host.bmmc_cache_attention(_attention(**between), k, v, 1 << 40, need, None) == ALIAS
    rows = dict(out_head=64 + 40, out_token=8 * 104, table_stride=104 // 2, table=B + 128)
    assert host.bmmc_cache_attention(_attention(**rows), k, v, 1 << 40, need, None) == ACCEPTED
    rows["table_width"] = 21
    assert host.bmmc_cache_attention(_attention(**rows), k, v, 1 << 40, 1 << 30, None) == ALIAS


def test_attention_workspace(host):
    a = _attention()
    need = host.bmmc_cache_attention_workspace(a)
    assert need > 0
    k, v = _cache(D), _cache(E)
    assert host.bmmc_cache_attention(a, k, v, 1 << 40, need, None) == ACCEPTED
    assert host.bmmc_cache_attention(a, k, v, 1 << 40, need - 1, None) == BAD
    assert host.bmmc_cache_attention(a, k, v, None, need, None) == BAD
    assert host.bmmc_cache_attention(a, k, v, (1 << 40) + 8, need, None) == BAD
    assert host.bmmc_cache_attention(a, k, v, B, need, None) == ALIAS  # out
    assert host.bmmc_cache_attention(a, k, v, D - need + 16, need, None) == ALIAS  # a cache
    assert host.bmmc_cache_attention(None, k, v, 1 << 40, need, None) == BAD
    assert host.bmmc_cache_attention(a, None, v, 1 << 40, need, None) == BAD
    assert host.bmmc_cache_attention_workspace(None) == -1
    assert host.bmmc_cache_attention_workspace(_attention(heads=3)) == -1
    assert host.bmmc_cache_attention_workspace(_attention(tokens=0)) == 0
    # one page is one part, and many rows are enough without parts
    assert host.bmmc_cache_attention_workspace(_attention(table_width=1)) == 0
    assert host.bmmc_cache_attention_workspace(_attention(tokens=1 << 20)) == 0


def test_workspaces_are_known_before_there_are_arrays(host):
    """A program may ask for the workspace's size before it has any array; with and without starts."""
    nothing = dict(q=None, out=None, table=None, lengths=None, q_token=-1, out_head=-1)
    for starts, batch in ((0, 3), (None, 10)):
        need = host.bmmc_cache_attention_workspace(_attention(starts=None if starts is None else C + 0x2000, batch=batch))
        assert need > 0
        some = None if starts is None else 4
        assert host.bmmc_cache_attention_workspace(_attention(**nothing, starts=some, batch=batch)) == need
    for changes in ({"table": None}, {"table": C + 2}):
        a = _attention(**changes)
        assert host.bmmc_cache_attention(a, _cache(D), _cache(E), 1 << 40, 1 << 30, None) == BAD
    assert host.bmmc_cache_attention(_attention(tokens=0, table=C + 2), _cache(D), _cache(E), None, 0, None) == BAD


def _heads(at, token=6 * 64, heads=2, dim=64, out=None, **changes):
    h = dict(heads=heads, in_batch=0, in_token=token, in_head=dim, out_batch=0, out_token=token, out_head=dim)
    h.update(changes)
    return tk.bmmc_heads(at, out, *[h[n] for n in ("heads", "in_batch", "in_token", "in_head", "out_batch",
                                                   "out_token", "out_head")])


def _narrow(data, scale, dim=64, heads=2, page=16, **changes):
    return _cache(data, dim, heads, page, tk.E4M3, **dict(dict(scale=scale, scale_page=page * heads,
                                                               scale_place=heads, scale_head=1), **changes))


TURN = tk.bmmc_rotation(None, A, None, 0, tk.I64, 1, 1, 32, 0, 0, 1.0)


def _quantize(host, k=None, v=None, q=None, kc=None, vc=None, rotation=None, **changes):
    p = 0x1000000
    a = dict(q=q, k=k or _heads(B), v=v or _heads(B + p), k_cache=kc or _narrow(C, D),
             v_cache=vc or _narrow(C + p, D + p), pages=100, page=16, table=E, batch=3, width=20, stride=20,
             sequences=E + p, positions=E + 2 * p, kind=tk.I64, rotation=rotation, tokens=10, k_dim=64, v_dim=64,
             type=tk.BF16, stream=None)
    a.update(changes)
    return host.bmmc_cache_quantize(*a.values())


def test_quantize_refusals(host):
    p = 0x1000000
    q = _heads(A, token=512, heads=8, out=A + p)
    for how, status in [
            ({}, ACCEPTED), ({"tokens": 0, "positions": None}, OK), ({"q": q}, BAD), ({"q": q, "rotation": TURN}, ACCEPTED),
            ({"rotation": TURN}, ACCEPTED), ({"tokens": -1}, BAD), ({"tokens": 1 << 31}, BAD), ({"k_dim": 0}, BAD),
            ({"v_dim": 513}, BAD), ({"type": tk.E4M3}, BAD), ({"kind": 5}, BAD), ({"positions": None}, BAD),
            ({"positions": E + 4}, BAD), ({"sequences": None}, ACCEPTED), ({"sequences": E + 2}, BAD), ({"table": None}, BAD),
            ({"pages": 0}, ACCEPTED), ({"page": 0}, BAD), ({"batch": -1}, BAD), ({"width": 1 << 31}, BAD), ({"stride": -1}, BAD),
            ({"k": _heads(None)}, BAD), ({"k": _heads(B + 1)}, BAD), ({"k": _heads(B, heads=3)}, BAD), ({"v": _heads(B, in_token=-1)}, BAD),
            ({"kc": _cache(C)}, BAD), ({"kc": _narrow(C, None)}, BAD), ({"kc": _narrow(C, D + 2)}, BAD), ({"vc": _narrow(None, D)}, BAD),
            # elements, and scales, lie apart from one another
            ({"kc": _narrow(C, D, head_stride=63)}, ALIAS), ({"kc": _narrow(C, D, scale_head=0)}, ALIAS),
            ({"kc": _narrow(C, D, scale_page=0)}, ALIAS), ({"vc": _narrow(C, D + p)}, ALIAS), ({"vc": _narrow(C + p, D)}, ALIAS),
            ({"vc": _narrow(C + p, D + 4)}, ALIAS), ({"kc": _narrow(C, C)}, ALIAS), ({"kc": _narrow(C, C + p)}, ALIAS), ({"vc": _narrow(C + p, C + 8)}, ALIAS),
            # both caches, and both scales, in one array: pages of keys, then of values
            ({"kc": _narrow(C, D, page_stride=4096, scale_page=64), "vc": _narrow(C + 2048, D + 128, page_stride=4096, scale_page=64)}, ACCEPTED),
            ({"kc": _narrow(C, D, page_stride=4096, scale_page=64), "vc": _narrow(C + 2047, D + 128, page_stride=4096, scale_page=64)}, ALIAS),
            # nothing that is read lies in a cache or among the scales
            ({"k": _heads(C + 64)}, ALIAS), ({"v": _heads(D + 64)}, ALIAS), ({"q": _heads(C, out=A), "rotation": TURN}, ALIAS),
            ({"q": _heads(A, out=D), "rotation": TURN}, ALIAS), ({"q": _heads(A, out=B), "rotation": TURN}, ALIAS),
            # queries in place between keys and values, and sharing an element with them
            ({"q": _heads(B + 256, out=B + 256), "v": _heads(B + 512), "rotation": TURN}, ACCEPTED),
            ({"q": _heads(B + 254, out=B + 254), "v": _heads(B + 512), "rotation": TURN}, ALIAS)]:
        assert _quantize(host, **how) == status, how
    many = tk.bmmc_rotation(None, A, None, 0, tk.I64, 1, 2, 32, 0, 0, 1.0)
    assert _quantize(host, rotation=many) == BAD  # two axes need positions of their own


def test_quantize_does_not_write_its_numbers(host):
    """The caches, their scales and the turned queries share no byte with the indexes, positions and
    frequencies, which may lie between a cache's rows."""
    p = 0x1000000
    data, scales, rows = 100 * 16 * 2 * 64, 100 * 16 * 2 * 4, 10 * 512 * 2
    written = {"k_cache": (C, data), "v_cache": (C + p, data), "k_scale": (D, scales), "v_scale": (D + p, scales),
               "q": (A + p, rows)}
    q = _heads(A, token=512, heads=8, out=A + p)

    def turn(positions=None, freqs=A + 4 * p, axes=None):
        return tk.bmmc_rotation(positions, freqs, axes, 10, tk.I64, 1, 2 if positions else 1, 32, 0, 0, 1.0)
    reads = [("table", 240, lambda at: dict(table=at)), ("sequences", 40, lambda at: dict(sequences=at)),
             ("positions", 80, lambda at: dict(positions=at)), ("turns", 160, lambda at: dict(rotation=turn(positions=at))),
             ("freqs", 256, lambda at: dict(rotation=turn(freqs=at))), ("axes", 128, lambda at: dict(rotation=turn(axes=at)))]
    for where, (start, size) in written.items():
        for name, n, how in reads:
            for at, status in ((start - n, ACCEPTED), (start - n + 8, ALIAS), (start + size // 2, ALIAS), (start + size - 8, ALIAS),
                               (start + size, ACCEPTED)):
                assert _quantize(host, **{"q": q, "rotation": turn(), **how(at)}) == status, (where, name, hex(at))
    # pages of keys with 64 bytes behind each
    kc = _narrow(C, D, page_stride=16 * 2 * 64 + 64)
    assert _quantize(host, kc=kc, sequences=C + 2048) == ACCEPTED
    assert _quantize(host, kc=kc, sequences=C + 2048 + 28) == ALIAS


def _read(host, k=None, v=None, kc=None, vc=None, **changes):
    p = 0x1000000
    a = dict(k=k or _heads(None, out=B), v=v or _heads(None, out=B + p), k_cache=kc or _cache(C),
             v_cache=vc or _cache(C + p), pages=100, page=16, table=E, batch=3, width=20, stride=20,
             sequences=E + p, positions=E + 2 * p, kind=tk.I64, tokens=10, k_dim=64, v_dim=64, type=tk.BF16, stream=None)
    a.update(changes)
    return host.bmmc_cache_read(*a.values())


def test_read_refusals(host):
    p = 0x1000000
    for how, status in [
            ({}, ACCEPTED), ({"tokens": 0, "positions": None}, OK), ({"tokens": -1}, BAD), ({"k_dim": 513}, BAD), ({"v_dim": 0}, BAD),
            ({"type": tk.E4M3}, BAD), ({"positions": None}, BAD), ({"sequences": None}, ACCEPTED), ({"table": None}, BAD),
            ({"k": _heads(None)}, BAD), ({"k": _heads(None, out=B + 1)}, BAD), ({"v": _heads(None, out=B, heads=1)}, BAD),
            ({"k": _heads(None, out=B, out_head=63)}, ALIAS), ({"v": _heads(None, out=B)}, ALIAS), ({"v": _heads(None, out=B + 256)}, ACCEPTED),
            ({"v": _heads(None, out=B + 254)}, ALIAS), ({"k": _heads(None, out=C)}, ALIAS), ({"kc": _cache(C, kind=tk.F16)}, BAD),
            ({"kc": _narrow(C, D)}, BAD), ({"kc": _narrow(C, D), "vc": _narrow(C + p, D)}, ACCEPTED),
            ({"kc": _narrow(C, B), "vc": _narrow(C + p, D)}, ALIAS), ({"vc": _cache(C)}, ACCEPTED)]:
        assert _read(host, **how) == status, how


def test_read_does_not_write_its_indexes(host):
    """The two results share no byte with the table, the sequences or the positions, which may lie
    between their heads."""
    p = 0x1000000
    size = 9 * 6 * 64 * 2 + 2 * 64 * 2
    for start in (B, B + p):
        for name, n in (("table", 240), ("sequences", 40), ("positions", 80)):
            for at, status in ((start - n, ACCEPTED), (start - n + 8, ALIAS), (start, ALIAS), (start + size - 8, ALIAS),
                               (start + size, ACCEPTED), (start + 256, ACCEPTED), (start + 248, ALIAS)):
                assert _read(host, **{name: at}) == status, (name, hex(at))


def test_balance_refusals(host):
    p = 0x1000000
    base = dict(logits=A, stride=64, type=tk.F32, e=64, experts=B, kind=tk.I64, tokens=100, choices=4, mask=C, loss=D,
                counts=D + p, slopes=D + 2 * p, work=E, bytes=1 << 24, stream=None)
    for how, status in [
            ({}, ACCEPTED), ({"mask": None}, ACCEPTED), ({"tokens": 0, "logits": None, "experts": None}, ACCEPTED), ({"tokens": -1}, BAD),
            ({"tokens": 1 << 30}, BAD), ({"e": 0}, BAD), ({"e": 2049}, BAD), ({"choices": 0}, BAD), ({"choices": 1025}, BAD), ({"type": tk.E4M3}, BAD),
            ({"kind": 2}, BAD), ({"stride": -1}, BAD), ({"stride": 0}, ACCEPTED), ({"logits": A + 2}, BAD), ({"experts": B + 4}, BAD), ({"experts": B + 4, "kind": tk.I32}, ACCEPTED),
            ({"loss": None}, BAD), ({"counts": D + 2}, BAD), ({"slopes": None}, BAD), ({"work": None}, BAD), ({"bytes": 100}, BAD),
            ({"loss": A + 4}, ALIAS), ({"counts": B}, ALIAS), ({"slopes": C}, ALIAS), ({"work": D}, ALIAS), ({"loss": D + p}, ALIAS)]:
        assert host.bmmc_expert_balance(*{**base, **how}.values()) == status, how
    assert host.bmmc_expert_balance_workspace(-1, 4) == -1 and host.bmmc_expert_balance_workspace(4, 2049) == -1
    need = host.bmmc_expert_balance_workspace(100, 64)
    assert host.bmmc_expert_balance(*{**base, "bytes": need}.values()) == ACCEPTED
    assert host.bmmc_expert_balance(*{**base, "bytes": need - 1}.values()) == BAD
    back = dict(grad=D, logits=A, stride=64, type=tk.F32, e=64, slopes=D + p, tokens=100, mask=C, out=B, out_stride=64, stream=None)
    for how, status in [
            ({}, ACCEPTED), ({"tokens": 0, "grad": None}, OK), ({"tokens": -1}, BAD), ({"e": 0}, BAD), ({"type": 9}, BAD), ({"grad": None}, BAD),
            ({"slopes": None}, BAD), ({"logits": None}, BAD), ({"out": None}, BAD), ({"out": B + 2}, BAD), ({"out_stride": 63}, BAD),
            ({"out": A}, ALIAS), ({"out": C}, ALIAS), ({"out": D}, ALIAS), ({"out_stride": 1 << 41}, BAD)]:
        assert host.bmmc_expert_balance_backward(*{**back, **how}.values()) == status, how


# --------------------------------------------------------------------------
# The Python calls' checks, which come before the device's
# --------------------------------------------------------------------------

F8 = torch.float8_e4m3fn


def _args(**changes):
    a = dict(q=torch.zeros(3, 4, 16), k_cache=torch.zeros(5, 8, 2, 16), v_cache=torch.zeros(5, 8, 2, 24),
             page_table=torch.zeros(3, 2, dtype=torch.int32), lengths=torch.ones(3, dtype=torch.int32))
    a.update(changes)
    return a


@pytest.mark.parametrize("changes", [
    {"q": torch.zeros(3, 64)}, {"q": torch.zeros(3, 4, 16, dtype=torch.float64)}, {"q": torch.zeros(3, 3, 16)}, {"q": torch.zeros(3, 4, 18)},
    {"q": torch.zeros(3, 4, 16).transpose(1, 2)}, {"q": torch.zeros(2, 4, 16)}, {"q": torch.zeros(3, 4, 16, dtype=torch.float16)}, {"q": 3},
    {"k_cache": torch.zeros(5, 8, 16)}, {"k_cache": torch.zeros(4, 8, 2, 16)}, {"k_cache": torch.zeros(5, 8, 2, 16).to(F8)},
    {"k_cache": torch.zeros(5, 8, 2, 16).to(F8), "v_cache": torch.zeros(5, 8, 2, 24).to(F8)}, {"k_scale": torch.ones(2)},
    {"k_cache": torch.zeros(5, 8, 2, 4), "q": torch.zeros(3, 4, 4)}, {"v_cache": torch.zeros(5, 8, 2, 7)}, {"v_cache": torch.zeros(5, 8, 2, 513)},
    {"page_table": torch.zeros(3, 2, dtype=torch.int64)}, {"page_table": torch.zeros(6, dtype=torch.int32)}, {"page_table": torch.zeros(2, 3, dtype=torch.int32).t()},
    {"lengths": torch.ones(3, dtype=torch.int64)}, {"lengths": torch.ones(2, dtype=torch.int32)}, {"starts": torch.zeros(3, dtype=torch.int32)},
    {"starts": torch.zeros(4, dtype=torch.int64)}, {"scale": 0.0}, {"scale": -1.0}, {"scale": float("nan")}, {"window": -1},
    {"out": torch.zeros(3, 4, 16)}, {"out": torch.zeros(3, 4, 24, dtype=torch.float16)}, {"out": torch.zeros(3, 24, 4).transpose(1, 2)},
    {"out": torch.zeros(3, 4, 24, requires_grad=True)}, {"q": torch.zeros(3, 4, 16, requires_grad=True)},
    {"v_cache": torch.zeros(5, 8, 2, 24, requires_grad=True)}], ids=str)
def test_attention_calls_refuse(changes):
    with pytest.raises((ValueError, TypeError)) as e:
        bm.cache_attention(**_args(**changes))
    assert "device tensors" not in str(e.value)


@pytest.mark.parametrize("scale", [torch.ones(3), torch.ones(2, dtype=torch.float64), torch.ones(5, 8, 3), torch.ones(1, 2),
                                   torch.ones(2, requires_grad=True)], ids=str)
def test_scales_are_checked(scale):
    caches = dict(k_cache=torch.zeros(5, 8, 2, 16).to(F8), v_cache=torch.zeros(5, 8, 2, 24).to(F8))
    for name in ("k_scale", "v_scale"):
        scales = {"k_scale": torch.ones(2), "v_scale": torch.ones(2), name: scale}
        with pytest.raises(ValueError) as e:
            bm.cache_attention(**_args(**caches, **scales))
        assert "device tensors" not in str(e.value)
    for fine in (torch.ones(()), torch.ones(1), torch.ones(2), torch.ones(4)[::2], torch.ones(5, 2, 8).transpose(1, 2)):
        with pytest.raises(ValueError, match="device tensors"):
            bm.cache_attention(**_args(**caches, k_scale=fine, v_scale=torch.ones(5, 8, 2)))


def _append(**changes):
    a = dict(k=torch.zeros(3, 2, 16), v=torch.zeros(3, 2, 24), k_cache=torch.zeros(5, 8, 2, 16).to(F8),
             v_cache=torch.zeros(5, 8, 2, 24).to(F8), k_scale=torch.ones(5, 8, 2), v_scale=torch.ones(5, 8, 2),
             page_table=torch.zeros(3, 2, dtype=torch.int32), positions=torch.zeros(3, dtype=torch.int64))
    a.update(changes)
    return a


FREQS = torch.ones(8)


@pytest.mark.parametrize("changes", [
    {"k": torch.zeros(3, 2, 16).double()}, {"k": torch.zeros(2, 2, 16)}, {"k": torch.zeros(3, 32)}, {"v": torch.zeros(3, 2, 24).half()}, {"v": torch.zeros(3, 1, 24)},
    {"k_cache": torch.zeros(5, 8, 2, 16)}, {"k_cache": torch.zeros(5, 8, 2, 18).to(F8)}, {"v_cache": torch.zeros(5, 8, 3, 24).to(F8)},
    {"k_scale": torch.ones(2)}, {"k_scale": torch.ones(5, 8, 2).half()}, {"v_scale": torch.ones(8, 5, 2)}, {"k_scale": torch.ones(5, 8, 2, requires_grad=True)},
    {"page_table": torch.zeros(3, 2)}, {"positions": torch.zeros(2, dtype=torch.int64)}, {"positions": torch.zeros(3)}, {"sequences": torch.zeros(3, dtype=torch.int64)},
    {"q": torch.zeros(3, 4, 16)}, {"axes": torch.zeros(8, dtype=torch.int32)}, {"freqs": FREQS, "q_out": torch.zeros(3, 4, 16)}, {"freqs": torch.ones(9)},
    {"freqs": FREQS, "q": torch.zeros(3, 4, 18)}, {"freqs": FREQS, "q": torch.zeros(3, 4, 16).half()}, {"freqs": FREQS, "q": torch.zeros(3, 4, 16), "q_out": torch.zeros(3, 2, 16)},
    {"freqs": torch.ones(8, requires_grad=True)}, {"k": torch.zeros(3, 2, 16, requires_grad=True)},
    {"freqs": FREQS, "q": torch.zeros(3, 4, 16), "q_out": torch.zeros(3, 4, 16, requires_grad=True)}], ids=str)
def test_quantize_calls_refuse(changes):
    with pytest.raises((ValueError, TypeError)) as e:
        bm.cache_quantize(**_append(**changes))
    assert "device tensors" not in str(e.value)


def _back(**changes):
    a = dict(k_cache=torch.zeros(5, 8, 2, 16), v_cache=torch.zeros(5, 8, 2, 24), page_table=torch.zeros(3, 2, dtype=torch.int32),
             positions=torch.zeros(3, dtype=torch.int64))
    a.update(changes)
    return a


@pytest.mark.parametrize("changes", [
    {"k_cache": torch.zeros(5, 8, 2, 16).to(F8)}, {"k_cache": torch.zeros(5, 8, 2, 16).to(F8), "v_cache": torch.zeros(5, 8, 2, 24).to(F8), "k_scale": torch.ones(2), "v_scale": torch.ones(2)},
    {"dtype": torch.float16}, {"dtype": F8}, {"dtype": torch.float64}, {"dtype": "float32"}, {"k_scale": torch.ones(2)}, {"v_cache": torch.zeros(5, 8, 3, 24)},
    {"positions": torch.zeros((), dtype=torch.int64)}, {"positions": torch.zeros(3)}, {"sequences": torch.zeros(2, dtype=torch.int32)}, {"page_table": torch.zeros(6, dtype=torch.int32)},
    {"k_out": torch.zeros(3, 2, 24)}, {"v_out": torch.zeros(3, 2, 24).half()}, {"v_out": torch.zeros(3, 24, 2).transpose(1, 2)}, {"k_out": torch.zeros(3, 2, 16, requires_grad=True)},
    {"k_cache": torch.zeros(5, 8, 2, 16, requires_grad=True)}], ids=str)
def test_read_calls_refuse(changes):
    with pytest.raises((ValueError, TypeError)) as e:
        bm.cache_read(**_back(**changes))
    assert "device tensors" not in str(e.value)


CHOSEN = torch.zeros(3, 2, dtype=torch.int64)


@pytest.mark.parametrize("call", [
    lambda: bm.expert_balance(torch.zeros(3, 4).double(), CHOSEN), lambda: bm.expert_balance(torch.zeros(12), CHOSEN), lambda: bm.expert_balance(torch.zeros(3, 2049), CHOSEN),
    lambda: bm.expert_balance(torch.zeros(4, 3).t(), CHOSEN), lambda: bm.expert_balance(torch.zeros(2, 4), CHOSEN), lambda: bm.expert_balance(torch.zeros(3, 4), CHOSEN.float()),
    lambda: bm.expert_balance(torch.zeros(3, 4), CHOSEN.t().contiguous().t()), lambda: bm.expert_balance(torch.zeros(3, 4), CHOSEN[:, :0]), lambda: bm.expert_balance(torch.zeros(3, 4), CHOSEN.reshape(-1)),
    lambda: bm.expert_balance(torch.zeros(3, 4), CHOSEN, mask=torch.ones(3)), lambda: bm.expert_balance(torch.zeros(3, 4), CHOSEN, mask=torch.ones(2, dtype=torch.bool)),
    lambda: bm.expert_balance_backward(torch.ones(()), torch.zeros(3, 4), torch.ones(3)), lambda: bm.expert_balance_backward(torch.ones(2), torch.zeros(3, 4), torch.ones(4)),
    lambda: bm.expert_balance_backward(torch.ones(()).half(), torch.zeros(3, 4), torch.ones(4)), lambda: bm.expert_balance_backward(torch.ones((), requires_grad=True), torch.zeros(3, 4), torch.ones(4)),
    lambda: bm.expert_balance_backward(torch.ones(()), torch.zeros(3, 4), torch.ones(4, requires_grad=True)), lambda: bm.expert_balance_backward(torch.ones(()), torch.zeros(3, 4), torch.ones(4), out=torch.zeros(3, 5)),
    lambda: bm.expert_balance_backward(torch.ones(()), torch.zeros(3, 4), torch.ones(4), out=torch.zeros(3, 4, requires_grad=True))])
def test_balance_calls_refuse(call):
    with pytest.raises((ValueError, TypeError)) as e:
        call()
    assert "device tensors" not in str(e.value)


def test_host_tensors_are_refused():
    for call in (lambda: bm.cache_attention(**_args()), lambda: bm.cache_quantize(**_append()), lambda: bm.cache_read(**_back()),
                 lambda: bm.expert_balance(torch.zeros(3, 4), CHOSEN), lambda: bm.expert_balance(torch.zeros(3, 4, requires_grad=True), CHOSEN),
                 lambda: bm.expert_balance_backward(torch.ones(()), torch.zeros(3, 4), torch.ones(4)),
                 lambda: bm.cache_attention(**_args(), stream=5)):
        with pytest.raises(ValueError, match="device tensors"):
            call()


def test_tangents_are_refused():
    import torch.autograd.forward_ad as fwd
    with fwd.dual_level():
        for call in (lambda: bm.cache_attention(**_args(q=fwd.make_dual(torch.zeros(3, 4, 16), torch.ones(3, 4, 16)))),
                     lambda: bm.expert_balance(fwd.make_dual(torch.zeros(3, 4), torch.ones(3, 4)), CHOSEN),
                     lambda: bm.cache_read(**_back(k_cache=fwd.make_dual(torch.zeros(5, 8, 2, 16), torch.ones(5, 8, 2, 16)))),
                     lambda: bm.cache_quantize(**_append(k=fwd.make_dual(torch.zeros(3, 2, 16), torch.ones(3, 2, 16))))):
            with pytest.raises(ValueError, match="forward-mode"):
                call()
