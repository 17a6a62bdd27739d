"""CPU tests of the calls on token rows: exports, argument checks of the C
entry points and of the Python calls, and the host side of the kernels'
indexing.  No GPU call is made: accepted arguments are only tried on a build
whose launchers are stand-ins."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest

torch = pytest.importorskip("torch")

import bmmc_affine_index_amd as bm  # noqa: E402
from bmmc_affine_index_amd import tokens as tk  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TESTS = os.path.join(ROOT, "tests")
CSRC = os.path.join(ROOT, "bmmc_affine_index_amd", "csrc")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
INCLUDE = ["-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I" + os.path.join(ROOT, "include")]
SANITIZE = ["-fsanitize=address,undefined", "-fno-sanitize-recover=undefined"]
ACCEPTED = bm.ERR_HIP  # what the stand-in launchers return


def test_library_exports_every_header_function():
    header = open(os.path.join(ROOT, "include", "bmmc_tokens.h")).read()
    names = set(re.findall(r"^\S[^;()]*?\b(bmmc_\w+)\s*\(", header, flags=re.M))
    assert names == set(tk.TOKENS_EXPORTED)
    L = tk.tokens_lib()
    for name in names:
        assert hasattr(L, name), name


def test_struct_layouts_match_header(tmp_path):
    structs = {c.__name__: c for c in (tk.bmmc_heads, tk.bmmc_rotation, tk.bmmc_paged_cache)}
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "bmmc_tokens.h"',
             "int main(void) {"]
    for name, cls in structs.items():
        lines.append('printf("%s %%zu\\n", sizeof(%s));' % (name, name))
        for field, _ in cls._fields_:
            lines.append('printf("%s.%s %%zu\\n", offsetof(%s, %s));' % (name, field, name, field))
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines + ["return 0; }"]))
    exe = tmp_path / "layout"
    subprocess.check_call(["gcc", "-I" + os.path.join(ROOT, "include"), str(src), "-o", str(exe)])
    out = dict(l.split() for l in subprocess.check_output([str(exe)]).decode().splitlines())
    for name, cls in structs.items():
        assert int(out[name]) == ctypes.sizeof(cls), name
        for field, _ in cls._fields_:
            assert int(out[name + "." + field]) == getattr(cls, field).offset, (name, field)


@pytest.mark.skipif(shutil.which("g++") is None or bool(os.environ.get("LD_PRELOAD")),
                    reason="needs g++, and no library preloaded before the sanitizer's")
def test_host_side_of_the_indexing(tmp_path):
    exe = str(tmp_path / "host")
    subprocess.run(["g++", "-std=c++17", "-O1", "-g", *SANITIZE, *INCLUDE,
                    os.path.join(TESTS, "tokens_host.cpp"), "-L/opt/rocm/lib", "-lamdhip64",
                    "-Wl,-rpath,/opt/rocm/lib", "-o", exe], check=True, timeout=300)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0"))
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout + r.stderr


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="needs hipcc")
@pytest.mark.parametrize("src", ["order.hip", "experts.hip", "rotary.hip"])
def test_every_kernel_has_a_body(src, tmp_path):
    """Undefined behaviour can leave a kernel without instructions, which a
    wave would run past; every kernel ends in s_endpgm and none spills vector
    registers."""
    out = tmp_path / (src + ".s")
    subprocess.run([HIPCC, "-O3", "-std=c++17", "-I" + os.path.join(ROOT, "include"),
                    "--offload-arch=gfx950", "-Xclang", "-target-feature", "-Xclang",
                    "-packed-fp32-ops", "--cuda-device-only", "-S", "-o", str(out),
                    os.path.join(CSRC, "tokens", src)],
                   check=True, capture_output=True, timeout=600)
    s = out.read_text()
    kernels = re.findall(r"^\s*\.amdhsa_kernel\s+(\S+)", s, flags=re.M)
    assert kernels
    for name in kernels:
        start = s.index("\n%s:" % name)
        ins = [l.strip() for l in s[start:s.index(".Lfunc_end", start)].splitlines()[1:]]
        assert any(l.startswith("s_endpgm") for l in ins), name
    assert set(re.findall(r"\.vgpr_spill_count:\s*(\d+)", s)) == {"0"}


# --------------------------------------------------------------------------
# The C entry points' checks, on a build whose launchers are stand-ins
# --------------------------------------------------------------------------

@pytest.fixture(scope="module")
def host(tmp_path_factory):
    if shutil.which("g++") is None or not os.path.exists("/opt/rocm/lib"):
        pytest.skip("needs g++ and the ROCm runtime library")
    so = str(tmp_path_factory.mktemp("host") / "libtokens_host.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-fsanitize=undefined",
                    "-fno-sanitize-recover=undefined", *INCLUDE,
                    os.path.join(CSRC, "tokens", "api.cpp"), os.path.join(TESTS, "token_stubs.cpp"),
                    "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib", "-o", so],
                   check=True, timeout=300)
    L = ctypes.CDLL(so)
    real = tk.tokens_lib()
    for name in tk.TOKENS_EXPORTED:
        getattr(L, name).argtypes = getattr(real, name).argtypes
        getattr(L, name).restype = getattr(real, name).restype
    return L


A, B, C, D, E, G = (0x10000000 * k for k in range(1, 7))  # addresses nothing is read from


def _with(base, changes):
    args = dict(base)
    args.update(changes)
    return list(args.values())


@pytest.mark.parametrize("n,e,align,rows", [(0, 1, 1, 0), (10, 4, 1, 10), (10, 4, 16, 70),
                                            (3, 64, 16, 48), (1 << 20, 2048, 128, (1 << 20) + 2048 * 127),
                                            (-1, 4, 1, -1), (1 << 31, 4, 1, -1), (4, 0, 1, -1),
                                            (4, 2049, 1, -1), (4, 4, 0, -1), (4, 4, 1 << 31, -1),
                                            (4, 4, (1 << 31) - 1, -1)])
def test_rows_of_an_order(n, e, align, rows):
    assert tk.tokens_lib().bmmc_expert_rows(n, e, align) == rows


ORDER = dict(experts=A, kind=tk.I64, n=100000, e=8, align=1, offsets=B, counts=C, rows=D, slots=E,
             work=G, bytes=1 << 30, stream=None)


@pytest.mark.parametrize("changes,status", [
    ({}, ACCEPTED), ({"n": 0, "experts": None, "rows": None, "slots": None}, ACCEPTED),
    ({"n": 4096, "work": None, "bytes": 0}, ACCEPTED),
    ({"n": -1}, bm.ERR_INVALID_ARG), ({"n": 1 << 31}, bm.ERR_INVALID_ARG),
    ({"e": 0}, bm.ERR_INVALID_ARG), ({"e": 2049}, bm.ERR_INVALID_ARG),
    ({"align": 0}, bm.ERR_INVALID_ARG), ({"align": 1 << 30}, bm.ERR_INVALID_ARG),
    ({"kind": 2}, bm.ERR_INVALID_ARG), ({"experts": None}, bm.ERR_INVALID_ARG),
    ({"experts": A + 4}, bm.ERR_INVALID_ARG), ({"kind": tk.I32, "experts": A + 4}, ACCEPTED),
    ({"offsets": None}, bm.ERR_INVALID_ARG), ({"counts": C + 1}, bm.ERR_INVALID_ARG),
    ({"rows": None}, bm.ERR_INVALID_ARG), ({"slots": None}, bm.ERR_INVALID_ARG),
    ({"work": None}, bm.ERR_INVALID_ARG), ({"bytes": 8}, bm.ERR_INVALID_ARG)])
def test_order_refusals(host, changes, status):
    assert host.bmmc_expert_order(*_with(ORDER, changes)) == status


GATHER = dict(x=A, x_stride=100, rows=B, slots=C, tokens=10, choices=4, capacity=40, dim=100,
              kind=tk.BF16, out=D, out_stride=100, stream=None)


@pytest.mark.parametrize("changes,status", [
    ({}, ACCEPTED), ({"x": A + 2}, ACCEPTED), ({"x_stride": 0}, ACCEPTED),
    ({"tokens": 0, "capacity": 0}, bm.OK), ({"tokens": 0, "x": None, "rows": None}, ACCEPTED),
    ({"capacity": 0}, bm.ERR_INVALID_ARG), ({"tokens": -1}, bm.ERR_INVALID_ARG),
    ({"tokens": 1 << 30}, bm.ERR_INVALID_ARG), ({"choices": 0}, bm.ERR_INVALID_ARG),
    ({"choices": 1025}, bm.ERR_INVALID_ARG), ({"dim": 0}, bm.ERR_INVALID_ARG),
    ({"dim": 1 << 31}, bm.ERR_INVALID_ARG), ({"kind": tk.E4M3}, bm.ERR_INVALID_ARG),
    ({"kind": -1}, bm.ERR_INVALID_ARG), ({"x": None}, bm.ERR_INVALID_ARG),
    ({"x": A + 1}, bm.ERR_INVALID_ARG), ({"kind": tk.F32, "out": D + 2}, bm.ERR_INVALID_ARG),
    ({"rows": None}, bm.ERR_INVALID_ARG), ({"slots": None}, bm.ERR_INVALID_ARG),
    ({"x_stride": -100}, bm.ERR_INVALID_ARG), ({"out_stride": 99}, bm.ERR_INVALID_ARG),
    ({"x_stride": 1 << 50}, bm.ERR_INVALID_ARG), ({"out": A}, bm.ERR_ALIAS),
    ({"out": A + 10 * 200 - 2}, bm.ERR_ALIAS), ({"out": A + 10 * 200}, ACCEPTED),
    ({"x": D + 40 * 200 - 2}, bm.ERR_ALIAS), ({"x": D + 40 * 200}, ACCEPTED)])
def test_gather_refusals(host, changes, status):
    assert host.bmmc_expert_gather(*_with(GATHER, changes)) == status


COMBINE = dict(x=A, x_stride=100, rows=B, weights=C, wkind=tk.F32, tokens=10, choices=4,
               capacity=40, dim=100, kind=tk.F16, out=D, out_stride=100, stream=None)


@pytest.mark.parametrize("changes,status", [
    ({}, ACCEPTED), ({"weights": None}, ACCEPTED), ({"wkind": tk.F16}, ACCEPTED),
    ({"tokens": 0}, bm.OK), ({"capacity": 0}, bm.ERR_INVALID_ARG),
    ({"wkind": tk.BF16}, bm.ERR_INVALID_ARG), ({"weights": C + 2}, bm.ERR_INVALID_ARG),
    ({"x": None}, bm.ERR_INVALID_ARG), ({"out": None}, bm.ERR_INVALID_ARG),
    ({"rows": B + 2}, bm.ERR_INVALID_ARG), ({"out_stride": 0}, bm.ERR_INVALID_ARG),
    ({"tokens": 1, "out_stride": 0}, ACCEPTED), ({"out": A}, bm.ERR_ALIAS)])
def test_combine_refusals(host, changes, status):
    assert host.bmmc_expert_combine(*_with(COMBINE, changes)) == status


BACKWARD = dict(grad=A, grad_stride=100, x=B, x_stride=100, rows=C, slots=D, weights=E,
                wkind=tk.F32, tokens=10, choices=4, capacity=40, dim=100, kind=tk.BF16,
                grad_in=G, grad_in_stride=100, grad_weights=G + (1 << 20), stream=None)


@pytest.mark.parametrize("changes,status", [
    ({}, ACCEPTED), ({"tokens": 0, "capacity": 0}, bm.OK), ({"capacity": 0}, bm.ERR_INVALID_ARG),
    ({"weights": None}, bm.ERR_INVALID_ARG), ({"grad_weights": None}, bm.ERR_INVALID_ARG),
    ({"grad": None}, bm.ERR_INVALID_ARG), ({"x": None}, bm.ERR_INVALID_ARG),
    ({"slots": None}, bm.ERR_INVALID_ARG), ({"grad_in": A}, bm.ERR_ALIAS),
    ({"grad_in": B}, bm.ERR_ALIAS), ({"grad_in_stride": 50}, bm.ERR_INVALID_ARG),
    ({"wkind": tk.F16}, bm.ERR_INVALID_ARG), ({"dim": 0}, bm.ERR_INVALID_ARG)])
def test_combine_backward_refusals(host, changes, status):
    assert host.bmmc_expert_combine_backward(*_with(BACKWARD, changes)) == status


def _heads(**changes):
    h = dict(x=A, out=B, heads=8, in_batch=0, in_token=1024, in_head=128, out_batch=0,
             out_token=1024, out_head=128)
    h.update(changes)
    return tk.bmmc_heads(*h.values())


def _turn(**changes):
    r = dict(positions=C, freqs=D, axis_of_pair=None, axis_stride=0, position_type=tk.I64,
             freqs_are_64=1, axes=1, pairs=64, interleaved=0, inverse=0, scale=1.0)
    r.update(changes)
    return tk.bmmc_rotation(*r.values())


@pytest.mark.parametrize("heads,turn,args,status", [
    ({}, {}, {}, ACCEPTED),
    ({"out": A}, {}, {}, ACCEPTED),                                   # in place
    ({"out": A, "out_token": 2048}, {}, {}, bm.ERR_ALIAS),            # in place, other strides
    ({"out": A + 256}, {}, {}, bm.ERR_ALIAS),
    ({"out_head": 64}, {}, {}, bm.ERR_ALIAS),                         # heads of the result overlap
    ({"out_token": 0}, {}, {}, bm.ERR_ALIAS),
    ({"in_head": 0}, {}, {}, ACCEPTED),                               # one head read for all
    ({"out_head": 1280, "out_token": 128}, {}, {}, ACCEPTED),         # heads before tokens
    ({"heads": 0}, {}, {}, bm.ERR_INVALID_ARG), ({"x": None}, {}, {}, bm.ERR_INVALID_ARG),
    ({"out": None}, {}, {}, bm.ERR_INVALID_ARG), ({"x": A + 1}, {}, {}, bm.ERR_INVALID_ARG),
    ({"in_token": -1}, {}, {}, bm.ERR_INVALID_ARG),
    ({}, {"pairs": 0}, {}, bm.ERR_INVALID_ARG), ({}, {"pairs": 65}, {}, bm.ERR_INVALID_ARG),
    ({}, {"axes": 0}, {}, bm.ERR_INVALID_ARG), ({}, {"axes": 9}, {}, bm.ERR_INVALID_ARG),
    ({}, {"positions": None}, {}, bm.ERR_INVALID_ARG), ({}, {"freqs": None}, {}, bm.ERR_INVALID_ARG),
    ({}, {"freqs": D + 4}, {}, bm.ERR_INVALID_ARG),
    ({}, {"freqs": D + 4, "freqs_are_64": 0}, {}, ACCEPTED),
    ({}, {"positions": C + 4}, {}, bm.ERR_INVALID_ARG),
    ({}, {"position_type": 3}, {}, bm.ERR_INVALID_ARG),
    ({}, {"axis_of_pair": E + 2}, {}, bm.ERR_INVALID_ARG),
    ({}, {}, {"tokens": 0}, bm.OK), ({}, {}, {"batch": 0}, bm.OK),
    ({}, {}, {"tokens": -1}, bm.ERR_INVALID_ARG),
    ({}, {}, {"batch": 1 << 16, "tokens": 1 << 16}, bm.ERR_INVALID_ARG),
    ({}, {}, {"dim": 513}, bm.ERR_INVALID_ARG), ({}, {}, {"dim": 0}, bm.ERR_INVALID_ARG),
    ({}, {}, {"kind": tk.E4M3}, bm.ERR_INVALID_ARG), ({}, {}, {"count": 3}, bm.ERR_INVALID_ARG),
    ({}, {}, {"count": 0}, bm.ERR_INVALID_ARG)])
def test_rotary_refusals(host, heads, turn, args, status):
    a = dict(count=1, batch=1, tokens=10, dim=128, kind=tk.BF16)
    a.update(args)
    h = (tk.bmmc_heads * 2)(_heads(**heads), _heads(x=E, out=G))
    r = _turn(**turn)
    assert host.bmmc_rotary(h, a["count"], a["batch"], a["tokens"], a["dim"], a["kind"],
                            ctypes.byref(r), None) == status


def test_rotary_of_two(host):
    """Views of one projection, in place, lie between one another; a result of
    its own must not lie in the other tensor."""
    wide = dict(in_token=2048, out_token=2048)

    def status(q, k):
        h = (tk.bmmc_heads * 2)(q, k)
        return host.bmmc_rotary(h, 2, 1, 10, 128, tk.BF16, ctypes.byref(_turn()), None)
    assert status(_heads(out=A, **wide), _heads(x=A + 2048, out=A + 2048, **wide)) == ACCEPTED
    assert status(_heads(out=A, **wide), _heads(x=A + 2048, out=A, **wide)) == bm.ERR_ALIAS
    assert status(_heads(out=B, **wide), _heads(x=B + 2048, out=C, **wide)) == bm.ERR_ALIAS
    assert status(_heads(out=B), _heads(x=E, out=G)) == ACCEPTED


WIDE = dict(in_token=2048, out_token=2048)  # 8 of the 16 heads of a projection's token


@pytest.mark.parametrize("q,k,status", [
    # the same heads turned in place and read for a result of their own
    (dict(out=A, **WIDE), dict(out=G, **WIDE), bm.ERR_ALIAS),
    # in place, four of eight heads in common; one element; the next token's first head
    (dict(out=A, **WIDE), dict(x=A + 1024, out=A + 1024, **WIDE), bm.ERR_ALIAS),
    (dict(out=A, **WIDE), dict(x=A + 2046, out=A + 2046, **WIDE), bm.ERR_ALIAS),
    (dict(out=A, **WIDE), dict(x=A + 2304, out=A + 2304, **WIDE), bm.ERR_ALIAS),
    # in place, and the other's token strides are not the same
    (dict(out=A, **WIDE), dict(x=A + 2048, out=A + 2048), bm.ERR_ALIAS),
    # read only by the other: between its tokens, and not quite
    (dict(out=A, **WIDE), dict(x=A + 2048, out=G, **WIDE), ACCEPTED),
    (dict(out=A, **WIDE), dict(x=A + 2050, out=G, **WIDE), bm.ERR_ALIAS),
    (dict(out=A, **WIDE), dict(x=A + 2048, out=G, in_token=0), ACCEPTED),
    (dict(out=A, **WIDE), dict(x=A, out=G, in_token=0, in_head=0), bm.ERR_ALIAS),
    # every second head, and head by head before the tokens
    (dict(out=A, in_head=256, out_head=256, **WIDE),
     dict(x=A + 256, out=A + 256, in_head=256, out_head=256, **WIDE), ACCEPTED),
    (dict(out=A, in_head=256, out_head=256, **WIDE),
     dict(x=A + 254, out=A + 254, in_head=256, out_head=256, **WIDE), bm.ERR_ALIAS),
    (dict(out=A, in_token=128, out_token=128, in_head=1280, out_head=1280),
     dict(x=A + 8 * 2560, out=A + 8 * 2560, in_token=128, out_token=128, in_head=1280,
          out_head=1280), ACCEPTED),
    (dict(out=A, in_token=128, out_token=128, in_head=1280, out_head=1280),
     dict(x=A + 7 * 2560, out=A + 7 * 2560, in_token=128, out_token=128, in_head=1280,
          out_head=1280), bm.ERR_ALIAS)])
def test_rotary_of_two_that_share_heads(host, q, k, status):
    """What one tensor reads, another turned in place must not write."""
    for pair in ((q, k), (k, q)):
        h = (tk.bmmc_heads * 2)(*(_heads(**p) for p in pair))
        assert host.bmmc_rotary(h, 2, 1, 10, 128, tk.BF16, ctypes.byref(_turn()), None) == status


def test_rotary_of_two_in_batches(host):
    """Views of [batch, tokens, heads, size] and [batch, heads, tokens, size]."""
    def status(at, **strides):
        s = dict({d + n: v for n, v in strides.items() for d in ("in_", "out_")})
        h = (tk.bmmc_heads * 2)(_heads(out=A, **s), _heads(x=A + at, out=A + at, **s))
        return host.bmmc_rotary(h, 2, 6, 10, 128, tk.BF16, ctypes.byref(_turn()), None)
    flat = dict(batch=10 * 2048, token=2048, head=128)
    assert status(2048, **flat) == ACCEPTED and status(2046, **flat) == bm.ERR_ALIAS
    loose = dict(batch=10 * 2048 + 999, token=2048, head=128)  # tokens of two entries not in step
    assert status(2048, **loose) == ACCEPTED and status(2050, **loose) == bm.ERR_ALIAS
    first = dict(batch=16 * 1280, token=128, head=1280)
    assert status(8 * 2560, **first) == ACCEPTED and status(8 * 2560 - 2, **first) == bm.ERR_ALIAS
    inside = dict(batch=128, token=6 * 2048, head=6 * 128)  # the batch within a token's heads
    assert status(8 * 6 * 256, **inside) == ACCEPTED and status(7 * 6 * 256, **inside) == bm.ERR_ALIAS


def test_shared_elements_by_counting(host):
    """Small arrays at random: refused where an element that one tensor turned in
    place writes is one that the other reads or writes, and only there."""
    import itertools
    import random
    rng = random.Random(11)
    seen = {ACCEPTED: 0, bm.ERR_ALIAS: 0}

    def elements(at, strides, sizes):
        steps = itertools.product(*(range(n) for n in sizes))
        starts = [at + sum(i * s for i, s in zip(step, strides)) for step in steps]
        return [x + d for x in starts for d in range(2)]
    while min(seen.values()) < 400:
        sizes = [(rng.randint(1, 3), rng.randint(1, 4), rng.randint(1, 3)) for _ in range(2)]
        sizes[1] = sizes[0][:2] + sizes[1][2:]
        strides = [tuple(rng.choice([0, 2, 3, 4, 6, 8, 12, 13, 24, 48]) for _ in range(3))
                   for _ in range(2)]
        if rng.random() < 0.5:
            strides[1] = strides[0]
        at = [400, 400 + rng.randint(-30, 30)]
        mine, other = (elements(*t) for t in zip(at, strides, sizes))
        want = bm.ERR_ALIAS if set(mine) & set(other) else ACCEPTED
        names = ("batch", "token", "head")
        q, k = (dict({d + n: v for d in ("in_", "out_") for n, v in zip(names, s)},
                     x=A + 2 * t, out=A + 2 * t, heads=n[2]) for t, s, n in zip(at, strides, sizes))
        k.update(out=G, out_batch=100, out_token=20, out_head=2)

        def status(*pair):
            h = (tk.bmmc_heads * 2)(*(_heads(**p) for p in pair))
            return host.bmmc_rotary(h, len(pair), *sizes[0][:2], 2, tk.BF16,
                                    ctypes.byref(_turn(pairs=1)), None)
        if status(q) != ACCEPTED:
            continue  # heads of one result among each other's are refused for themselves
        assert len(set(mine)) == len(mine)
        assert status(q, k) == want and status(k, q) == want
        seen[want] += 1


def _cache(**changes):
    c = dict(data=E, scale=None, page_stride=16 * 1024, place_stride=1024, head_stride=128,
             scale_stride=0, kind=tk.BF16)
    c.update(changes)
    return tk.bmmc_paged_cache(*c.values())


APPEND = dict(pages=64, page_size=16, table=B, batch=4, width=16, stride=16, sequences=C,
              positions=D, pkind=tk.I64)
E4 = dict(kind=tk.E4M3, scale=A + (1 << 24))


@pytest.mark.parametrize("case,status", [
    ({}, ACCEPTED), ({"q": {}}, ACCEPTED), ({"turn": None}, ACCEPTED),
    ({"q": {"out": A + (1 << 26)}}, ACCEPTED),
    ({"tokens": 0}, bm.OK), ({"args": {"sequences": None}}, ACCEPTED),
    ({"args": {"batch": 0, "table": None}}, ACCEPTED), ({"args": {"pages": 0}}, ACCEPTED),
    ({"turn": {"positions": None}}, ACCEPTED),
    ({"turn": {"positions": None, "axes": 2}}, bm.ERR_INVALID_ARG),
    ({"turn": None, "q": {}}, bm.ERR_INVALID_ARG),
    ({"kc": E4, "vc": dict(E4, data=E + (1 << 24))}, ACCEPTED),
    ({"kc": E4}, bm.ERR_INVALID_ARG),                              # one 8-bit cache of two
    ({"kc": {"kind": tk.E4M3}, "vc": {"kind": tk.E4M3}}, bm.ERR_INVALID_ARG),  # no scale
    ({"kc": {"scale": A}}, bm.ERR_INVALID_ARG),                    # a scale without 8 bits
    ({"kc": dict(E4, scale_stride=2), "vc": E4}, bm.ERR_INVALID_ARG),
    ({"kc": {"kind": tk.F32}, "vc": {"kind": tk.F32}}, bm.ERR_INVALID_ARG),
    ({"kc": {"data": None}}, bm.ERR_INVALID_ARG), ({"kc": {"data": E + 1}}, bm.ERR_INVALID_ARG),
    ({"kc": {"head_stride": 64}}, bm.ERR_ALIAS),                   # heads overlap
    ({"kc": {"page_stride": 1024}}, bm.ERR_ALIAS),                 # pages overlap
    ({"kc": {"place_stride": 128, "head_stride": 2048}}, ACCEPTED),  # heads before places
    ({"kc": {"data": A}}, bm.ERR_ALIAS),                           # the keys lie in the cache
    ({"v": {"heads": 4}}, bm.ERR_INVALID_ARG), ({"k": {"x": None}}, bm.ERR_INVALID_ARG),
    ({"args": {"page_size": 0}}, bm.ERR_INVALID_ARG), ({"args": {"pages": -1}}, bm.ERR_INVALID_ARG),
    ({"args": {"table": None}}, bm.ERR_INVALID_ARG), ({"args": {"positions": None}}, bm.ERR_INVALID_ARG),
    ({"args": {"pkind": 2}}, bm.ERR_INVALID_ARG), ({"args": {"batch": -1}}, bm.ERR_INVALID_ARG),
    ({"args": {"sequences": C + 1}}, bm.ERR_INVALID_ARG),
    ({"args": {"stride": -16}}, bm.ERR_INVALID_ARG),
    ({"k_dim": 0}, bm.ERR_INVALID_ARG), ({"k_dim": 513}, bm.ERR_INVALID_ARG),
    ({"k_dim": 100}, bm.ERR_INVALID_ARG),                          # 64 pairs do not fit
    ({"tokens": -1}, bm.ERR_INVALID_ARG), ({"kind": tk.E4M3}, bm.ERR_INVALID_ARG)])
def test_append_refusals(host, case, status):
    args = dict(APPEND)
    args.update(case.get("args", {}))
    k, v = _heads(**case.get("k", {})), _heads(x=A + (1 << 22), **case.get("v", {}))
    q = _heads(x=A + (1 << 23), **case["q"]) if "q" in case else None
    if q is not None and "out" not in case["q"]:
        q.out = G
    turn = case.get("turn", {})
    turn = None if turn is None else _turn(**turn)
    kc, vc = _cache(**case.get("kc", {})), _cache(**{"data": E + (1 << 26), **case.get("vc", {})})
    assert host.bmmc_cache_append(q, k, v, kc, vc, *args.values(), turn, case.get("tokens", 10),
                                  case.get("k_dim", 128), 128, case.get("kind", tk.BF16),
                                  None) == status


def test_two_caches_in_one_array(host):
    """Keys and values of a page next to each other: [pages, 2, places, heads, size]."""
    k, v = _heads(), _heads(x=A + (1 << 22))
    kc = _cache(page_stride=2 * 16 * 1024)
    vc = _cache(page_stride=2 * 16 * 1024, data=E + 16 * 1024 * 2)
    assert host.bmmc_cache_append(None, k, v, kc, vc, *APPEND.values(), None, 10, 128, 128,
                                  tk.BF16, None) == ACCEPTED


VAL = A + 2048 + 1024  # the values of a token with 8 heads of queries and 4 of keys before them


@pytest.mark.parametrize("q,k,v,status", [
    (dict(), dict(x=A + 2048), dict(x=VAL), ACCEPTED),        # views of one projection
    (dict(), dict(x=A), dict(x=VAL), bm.ERR_ALIAS),           # the queries are the keys
    (dict(), dict(x=A + 2048), dict(x=A), bm.ERR_ALIAS),
    (dict(), dict(x=A + 2046), dict(x=VAL), bm.ERR_ALIAS),
    (dict(), dict(x=A + 2048), dict(x=VAL + 2), bm.ERR_ALIAS),  # the next token's first query
    (dict(), dict(x=A + 2048), dict(x=A + 1024), bm.ERR_ALIAS),
    (dict(), dict(x=A + 2048, in_token=0), dict(x=A + 2560, in_token=0), ACCEPTED),
    (dict(), dict(x=A + 4096, in_token=0), dict(x=VAL), bm.ERR_ALIAS),
    # a result of its own keeps clear of both
    (dict(out=G), dict(x=A), dict(x=A), ACCEPTED),
    (dict(out=B), dict(x=B + 2048), dict(x=VAL), bm.ERR_ALIAS)])
def test_append_of_queries_in_place(host, q, k, v, status):
    """Queries turned in place share no elements with the keys and values that
    are read in the same pass."""
    token = dict(in_token=2048, out_token=2048)
    q, k, v = (_heads(**{"out": A, **token, "heads": n, **h}) for h, n in ((q, 8), (k, 4), (v, 4)))
    args = {**APPEND, "table": D + (1 << 20)}
    kc, vc = _cache(), _cache(data=E + (1 << 26))
    assert host.bmmc_cache_append(q, k, v, kc, vc, *args.values(), _turn(), 10, 128, 128, tk.BF16,
                                  None) == status


PLACE = 8 * 256  # elements of a place that holds both a key and a value of 8 heads


@pytest.mark.parametrize("kc,vc,status", [
    (dict(), dict(data=E), bm.ERR_ALIAS),                        # one cache for both
    (dict(), dict(data=E + 63 * 16 * 2048 + 32766), bm.ERR_ALIAS),  # its last element
    (dict(), dict(data=E + 64 * 16 * 2048), ACCEPTED),
    # keys and values of a place, and of a head, next to each other
    (dict(place_stride=PLACE, page_stride=16 * PLACE),
     dict(place_stride=PLACE, page_stride=16 * PLACE, data=E + PLACE), ACCEPTED),
    (dict(place_stride=PLACE, page_stride=16 * PLACE),
     dict(place_stride=PLACE, page_stride=16 * PLACE, data=E + PLACE - 2), bm.ERR_ALIAS),
    (dict(place_stride=PLACE, page_stride=16 * PLACE, head_stride=256),
     dict(place_stride=PLACE, page_stride=16 * PLACE, head_stride=256, data=E + 256), ACCEPTED),
    (dict(place_stride=PLACE, page_stride=16 * PLACE, head_stride=256),
     dict(place_stride=PLACE, page_stride=16 * PLACE, head_stride=256, data=E + 254), bm.ERR_ALIAS),
    # keys before values in one layout, the other way round in the other: pages in common
    (dict(page_stride=32 * 1024), dict(page_stride=16 * 1024, data=E + 16 * 2048), bm.ERR_ALIAS),
    (dict(E4, head_stride=256, place_stride=PLACE, page_stride=16 * PLACE),
     dict(E4, head_stride=256, place_stride=PLACE, page_stride=16 * PLACE, data=E + 128), ACCEPTED),
    (dict(E4), dict(E4, data=E + 16), bm.ERR_ALIAS)])
def test_caches_that_share_elements(host, kc, vc, status):
    """A key and a value never go to one address."""
    def call(pages):
        args = {**APPEND, "pages": pages}
        return host.bmmc_cache_append(None, _heads(), _heads(x=A + (1 << 22)), _cache(**kc),
                                      _cache(**vc), *args.values(), None, 10, 128, 128, tk.BF16, None)
    assert call(64) == status
    assert call(0) == ACCEPTED  # caches without pages share nothing


# --------------------------------------------------------------------------
# The Python calls' checks
# --------------------------------------------------------------------------

def _order(tokens=4, choices=2, rows=None):
    rows = tokens * choices if rows is None else rows
    i = torch.int32
    return bm.ExpertOrder(torch.zeros(4, dtype=i), torch.zeros(3, dtype=i),
                          torch.zeros(tokens, choices, dtype=i), torch.zeros(rows, dtype=i))


BF = torch.bfloat16


@pytest.mark.parametrize("call", [
    lambda: bm.expert_order(torch.zeros(4, 2), 3),
    lambda: bm.expert_order(torch.zeros(4, 4, dtype=torch.int32)[:, :2], 3),
    lambda: bm.expert_order(torch.zeros(4, 2, dtype=torch.int64), 0),
    lambda: bm.expert_order(torch.zeros(4, 2, dtype=torch.int64), 2049),
    lambda: bm.expert_order(torch.zeros(4, 2, dtype=torch.int64), 3, align=0),
    lambda: bm.expert_gather(torch.zeros(4, 8), None),
    lambda: bm.expert_gather(torch.zeros(5, 8), _order()),
    lambda: bm.expert_gather(torch.zeros(4, 8, dtype=torch.float64), _order()),
    lambda: bm.expert_gather(torch.zeros(8, 4).t(), _order()),
    lambda: bm.expert_gather(torch.zeros(4, 0), _order()),
    lambda: bm.expert_gather(torch.zeros(4, 8), _order(rows=7)),
    lambda: bm.expert_gather(torch.zeros(4, 8), _order(), out=torch.zeros(8, 7)),
    lambda: bm.expert_gather(torch.zeros(4, 8), _order(), out=torch.zeros(8, 8, dtype=BF)),
    lambda: bm.expert_gather(torch.zeros(4, 8, requires_grad=True), _order(), out=torch.zeros(8, 8)),
    lambda: bm.expert_combine(torch.zeros(7, 8), _order()),
    lambda: bm.expert_combine(torch.zeros(8, 8), _order(), torch.zeros(4, 3)),
    lambda: bm.expert_combine(torch.zeros(8, 8), _order(), torch.zeros(4, 2, dtype=BF)),
    lambda: bm.expert_combine(torch.zeros(8, 8), _order(), torch.zeros(2, 4).t()),
    lambda: bm.expert_combine_backward(torch.zeros(4, 7), torch.zeros(8, 8), _order(), torch.zeros(4, 2)),
    lambda: bm.expert_combine_backward(torch.zeros(4, 8, dtype=BF), torch.zeros(8, 8), _order(),
                                       torch.zeros(4, 2)),
    lambda: bm.expert_gather_backward(torch.zeros(7, 8), _order()),
    lambda: bm.rotary_axes([]), lambda: bm.rotary_axes([-1, 2]), lambda: bm.rotary_axes([0]),
])
def test_expert_calls_refuse(call):
    with pytest.raises(ValueError):
        call()


POS = torch.zeros(4, dtype=torch.int64)
F = torch.ones(4, dtype=torch.float64)


@pytest.mark.parametrize("call", [
    lambda: bm.rotary(torch.zeros(4, 8), POS, F),
    lambda: bm.rotary(torch.zeros(4, 2, 8, dtype=torch.float64), POS, F),
    lambda: bm.rotary(torch.zeros(4, 2, 6), POS, F),
    lambda: bm.rotary(torch.zeros(4, 2, 514), POS, F),
    lambda: bm.rotary(torch.zeros(4, 0, 8), POS, F),
    lambda: bm.rotary(torch.zeros(4, 8, 2).transpose(1, 2), POS, F),
    lambda: bm.rotary(torch.zeros(4, 2, 8), POS.int()[:3], F),
    lambda: bm.rotary(torch.zeros(4, 2, 8), POS.float(), F),
    lambda: bm.rotary(torch.zeros(4, 2, 8), None, F),
    lambda: bm.rotary(torch.zeros(4, 2, 8), torch.zeros(9, 4, dtype=torch.int64), F),
    lambda: bm.rotary(torch.zeros(4, 2, 8), torch.zeros(4, 3, dtype=torch.int64).t(), F),
    lambda: bm.rotary(torch.zeros(4, 2, 8), POS, F.half()),
    lambda: bm.rotary(torch.zeros(4, 2, 8), POS, F[None]),
    lambda: bm.rotary(torch.zeros(4, 2, 8), POS, F, axes=torch.zeros(3, dtype=torch.int32)),
    lambda: bm.rotary(torch.zeros(4, 2, 8), POS, F, axes=torch.zeros(4, dtype=torch.int64)),
    lambda: bm.rotary((torch.zeros(4, 2, 8), torch.zeros(3, 2, 8)), POS, F),
    lambda: bm.rotary((torch.zeros(4, 2, 8), torch.zeros(4, 2, 8, dtype=BF)), POS, F),
    lambda: bm.rotary([torch.zeros(4, 2, 8)] * 3, POS, F),
    lambda: bm.rotary(torch.zeros(4, 2, 8), POS, F, out=torch.zeros(4, 2, 9)),
    lambda: bm.rotary(torch.zeros(4, 2, 8, requires_grad=True), POS, F, out=torch.zeros(4, 2, 8)),
])
def test_rotary_calls_refuse(call):
    with pytest.raises(ValueError):
        call()


def _append(**changes):
    a = dict(k=torch.zeros(4, 2, 8), v=torch.zeros(4, 2, 8), k_cache=torch.zeros(3, 4, 2, 8),
             v_cache=torch.zeros(3, 4, 2, 8), page_table=torch.zeros(4, 2, dtype=torch.int32),
             positions=POS)
    a.update(changes)
    return bm.cache_append(**a)


F8 = torch.float8_e4m3fn


@pytest.mark.parametrize("changes", [
    {"k": torch.zeros(4, 2, 8, dtype=BF)}, {"k": torch.zeros(5, 2, 8)}, {"k": torch.zeros(4, 8)},
    {"k_cache": torch.zeros(3, 4, 2, 9)}, {"k_cache": torch.zeros(3, 4, 2, 8, dtype=BF)},
    {"k_cache": torch.zeros(2, 4, 2, 8)}, {"k_cache": torch.zeros(3, 4, 8, 2).transpose(2, 3)},
    {"k_cache": torch.zeros(3, 4, 2, 8).to(F8)},
    {"k_scale": torch.ones(2)},
    {"k_cache": torch.zeros(3, 4, 2, 8).to(F8), "k_scale": torch.ones(3)},
    {"k_cache": torch.zeros(3, 0, 2, 8), "v_cache": torch.zeros(3, 0, 2, 8)},
    {"page_table": torch.zeros(4, 2, dtype=torch.int64)},
    {"page_table": torch.zeros(2, 4, dtype=torch.int32).t()},
    {"positions": POS[:3]}, {"positions": POS.float()},
    {"sequences": torch.zeros(4, dtype=torch.int64)}, {"sequences": torch.zeros(3, dtype=torch.int32)},
    {"q": torch.zeros(4, 2, 8)}, {"turns": POS}, {"q_out": torch.zeros(4, 2, 8)},
    {"freqs": F, "q": torch.zeros(4, 2, 6)}, {"freqs": F, "turns": POS[:2]},
    {"freqs": torch.ones(5)}, {"freqs": F, "q_out": torch.zeros(4, 2, 8)},
    {"k": torch.zeros(4, 2, 8, requires_grad=True)},
    {"k": torch.zeros(4, 2, 520), "v": torch.zeros(4, 2, 520)}])
def test_append_calls_refuse(changes):
    with pytest.raises(ValueError):
        _append(**changes)


def _asks(*shape, dtype=None):
    return torch.zeros(*shape, dtype=dtype, requires_grad=True)


WRITTEN = [  # calls that write into a tensor `t`, with its shape
    ((8, 8), lambda t: bm.expert_gather(torch.zeros(4, 8), _order(), out=t)),
    ((4, 8), lambda t: bm.expert_combine(torch.zeros(8, 8), _order(), out=t)),
    ((4, 8), lambda t: bm.expert_gather_backward(torch.zeros(8, 8), _order(), out=t)),
    ((4, 2, 8), lambda t: bm.rotary(torch.zeros(4, 2, 8), POS, F, out=t)),
    ((4, 2, 8), lambda t: bm.rotary((torch.zeros(4, 2, 8),) * 2, POS, F, out=(None, t))),
    ((4, 2, 8), lambda t: bm.rotary_backward(torch.zeros(4, 2, 8), POS, F, out=t)),
    ((4, 2, 8), lambda t: _append(freqs=F, q=torch.zeros(4, 2, 8), q_out=t)),
    ((3, 4, 2, 8), lambda t: _append(k_cache=t)), ((3, 4, 2, 8), lambda t: _append(v_cache=t))]


@pytest.mark.parametrize("shape,call", WRITTEN)
def test_tensors_that_ask_for_a_gradient_are_not_written(shape, call):
    with pytest.raises(ValueError, match="must not ask for a gradient"):
        call(_asks(*shape))
    with torch.no_grad(), pytest.raises(ValueError, match="device"):  # nothing else is wrong
        call(_asks(*shape))


@pytest.mark.parametrize("name,call", [
    ("freqs", lambda: bm.rotary(torch.zeros(4, 2, 8), POS, _asks(4))),
    ("freqs", lambda: bm.rotary(_asks(4, 2, 8), POS, _asks(4, dtype=torch.float64))),
    ("freqs", lambda: bm.rotary((torch.zeros(4, 2, 8), _asks(4, 2, 8)), POS, _asks(4))),
    ("freqs", lambda: bm.rotary_backward(torch.zeros(4, 2, 8), POS, _asks(4))),
    ("freqs", lambda: _append(freqs=_asks(4))),
    ("k_scale", lambda: _append(k_cache=torch.zeros(3, 4, 2, 8).to(F8), k_scale=_asks(2),
                                v_cache=torch.zeros(3, 4, 2, 8).to(F8), v_scale=torch.ones(2))),
    ("v_scale", lambda: _append(k_cache=torch.zeros(3, 4, 2, 8).to(F8), k_scale=torch.ones(1),
                                v_cache=torch.zeros(3, 4, 2, 8).to(F8), v_scale=_asks(1)))])
def test_gradients_that_are_not_made_are_refused(name, call):
    """There is no gradient of the frequencies or of a cache's scales."""
    with pytest.raises(ValueError, match=name + " has no gradient"):
        call()
    with torch.no_grad(), pytest.raises(ValueError, match="device"):  # nothing else is wrong
        call()


@pytest.mark.parametrize("call", [
    lambda: bm.expert_gather_backward(_asks(8, 8), _order()),
    lambda: bm.expert_combine_backward(_asks(4, 8), torch.zeros(8, 8), _order(), torch.zeros(4, 2)),
    lambda: bm.rotary_backward(_asks(4, 2, 8), POS, F),
    lambda: bm.rotary_backward((torch.zeros(4, 2, 8), _asks(4, 2, 8)), POS, F)])
def test_gradients_of_gradients_are_refused(call):
    with pytest.raises(ValueError, match="grad has no gradient"):
        call()
    with torch.no_grad(), pytest.raises(ValueError, match="device"):  # nothing else is wrong
        call()


def test_a_backward_call_takes_the_forward_pass_tensors():
    """Rows and weights that ask for a gradient are what a backward pass is
    for: only the device is wrong here."""
    with pytest.raises(ValueError, match="device"):
        bm.expert_combine_backward(torch.zeros(4, 8), _asks(8, 8), _order(), _asks(4, 2))


F8S = {n: torch.zeros(3, 4, 2, 8).to(F8) for n in ("k_cache", "v_cache")}
SCALES = {n: torch.ones(2) for n in ("k_scale", "v_scale")}


@pytest.mark.parametrize("shape,call", [
    ((4, 8), lambda t: bm.expert_gather(t, _order())),
    ((8, 8), lambda t: bm.expert_gather(torch.zeros(4, 8), _order(), out=t)),
    ((8, 8), lambda t: bm.expert_gather_backward(t, _order())),
    ((8, 8), lambda t: bm.expert_combine(t, _order())),
    ((8, 8), lambda t: bm.expert_combine(t, _order(), torch.zeros(4, 2))),
    ((4, 2), lambda t: bm.expert_combine(torch.zeros(8, 8), _order(), t)),
    ((4, 8), lambda t: bm.expert_combine(torch.zeros(8, 8), _order(), out=t)),
    ((4, 8), lambda t: bm.expert_combine_backward(t, torch.zeros(8, 8), _order(), torch.zeros(4, 2))),
    ((8, 8), lambda t: bm.expert_combine_backward(torch.zeros(4, 8), t, _order(), torch.zeros(4, 2))),
    ((4, 2), lambda t: bm.expert_combine_backward(torch.zeros(4, 8), torch.zeros(8, 8), _order(), t)),
    ((4, 2, 8), lambda t: bm.rotary(t, POS, F)), ((4, 2, 8), lambda t: bm.rotary(t, POS, F, out=t)),
    ((4, 2, 8), lambda t: bm.rotary((torch.zeros(4, 2, 8), t), POS, F)),
    ((4, 2, 8), lambda t: bm.rotary(torch.zeros(4, 2, 8), POS, F, out=t)),
    ((4, 2, 8), lambda t: bm.rotary_backward(t, POS, F)),
    ((4,), lambda t: bm.rotary(torch.zeros(4, 2, 8), POS, t)),
    ((4, 2, 8), lambda t: _append(k=t)), ((4, 2, 8), lambda t: _append(v=t)),
    ((3, 4, 2, 8), lambda t: _append(k_cache=t)), ((3, 4, 2, 8), lambda t: _append(v_cache=t)),
    ((4,), lambda t: _append(freqs=t)), ((4, 2, 8), lambda t: _append(freqs=F, q=t)),
    ((4, 2, 8), lambda t: _append(freqs=F, q=torch.zeros(4, 2, 8), q_out=t)),
    ((2,), lambda t: _append(**F8S, **{**SCALES, "k_scale": t})),
    ((2,), lambda t: _append(**F8S, **{**SCALES, "v_scale": t}))])
def test_tangents_are_refused(shape, call):
    """There is no forward-mode derivative: a dual tensor's tangent would be lost."""
    fw = torch.autograd.forward_ad
    with fw.dual_level():
        t = fw.make_dual(torch.zeros(shape), torch.ones(shape))
        for mode in (torch.enable_grad(), torch.no_grad()):
            with mode, pytest.raises(ValueError, match="forward-mode"):
                call(t)
    with pytest.raises(ValueError, match="device"):  # nothing else is wrong
        call(t)


def test_tangents_of_tensors_that_ask_for_a_gradient_are_refused():
    fw = torch.autograd.forward_ad
    with fw.dual_level():
        def dual(*shape, asks=True):
            return fw.make_dual(torch.zeros(shape, requires_grad=asks), torch.ones(shape))
        for call in (lambda: bm.expert_gather(dual(4, 8), _order()),
                     lambda: bm.expert_combine(dual(8, 8), _order()),
                     lambda: bm.expert_combine(_asks(8, 8), _order(), dual(4, 2, asks=False)),
                     lambda: bm.rotary((_asks(4, 2, 8), dual(4, 2, 8, asks=False)), POS, F),
                     lambda: bm.rotary(_asks(4, 2, 8), POS, dual(4, asks=False))):
            with pytest.raises(ValueError, match="forward-mode"):
                call()


def test_arrays_without_elements_have_no_strides_to_check():
    """An expanded gradient of no tokens: only the device is wrong."""
    none = torch.zeros(()).expand(0, 8)
    heads = torch.zeros(()).expand(0, 2, 8)
    order = _order(tokens=0)
    for call in (lambda: bm.expert_gather(none, order), lambda: bm.expert_combine(none, order),
                 lambda: bm.expert_gather_backward(none, order),
                 lambda: bm.expert_combine_backward(none, none, order, torch.zeros(0, 2)),
                 lambda: bm.rotary_backward(heads, POS[:0], F),
                 lambda: _append(k=heads, v=heads, positions=POS[:0])):
        with pytest.raises(ValueError, match="device"):
            call()


def test_host_tensors_are_refused():
    """Everything else in order: there is no path for host memory."""
    for call in (lambda: bm.expert_order(torch.zeros(4, 2, dtype=torch.int64), 3),
                 lambda: bm.expert_gather(torch.zeros(4, 8), _order()),
                 lambda: bm.expert_combine(torch.zeros(8, 8), _order(), torch.zeros(4, 2)),
                 lambda: bm.rotary(torch.zeros(4, 2, 8), POS, F), lambda: _append()):
        with pytest.raises(ValueError, match="device"):
            call()


def test_rotary_axes():
    assert bm.rotary_axes([2, 1, 1]).tolist() == [0, 0, 1, 2]
    assert bm.rotary_axes([1, 3, 2], interleaved=True).tolist() == [0, 1, 2, 1, 2, 1]


# --------------------------------------------------------------------------
# The native calls
# --------------------------------------------------------------------------

@pytest.mark.parametrize("call", [
    lambda n: n.order(), lambda n: n.order(torch.zeros(4, 2, dtype=torch.int64), 3, 1),
    lambda n: n.gather(1, 2, 3, 4, 5, 6), lambda n: n.order([[0, 1]], 3, 1, None),
    lambda n: n.order(torch.zeros(4, 2, dtype=torch.int64), "3", 1, None),
    lambda n: n.order(torch.zeros(4, 2, dtype=torch.int64), 2.5, 1, None),
    lambda n: n.combine(torch.zeros(8, 8), *_order()[2:], [1.0], None, None),
    lambda n: n.rotary((None,), POS, F, None, False, 1.0, None, False, None)])
def test_native_calls_count_and_type_their_arguments(call):
    with pytest.raises(TypeError):
        call(tk._calls())


@pytest.mark.parametrize("call", [
    lambda n: n.order(torch.zeros(4, 2, dtype=torch.int64), 1 << 40, 1, None),
    lambda n: n.order(torch.zeros(4, 2, dtype=torch.int64), -(1 << 40), 1, None),
    lambda n: n.order(torch.zeros(4, 2, dtype=torch.int64), (1 << 32) + 4, 1, None),
    lambda n: n.order(torch.zeros(4, 2, dtype=torch.int64), 4, 1 << 62, None),
    lambda n: n.rotary((), POS, F, None, False, 1.0, None, False, None)])
def test_native_calls_check_wide_numbers(call):
    with pytest.raises(ValueError):
        call(tk._calls())


def test_another_stream_needs_device_tensors():
    for call in (lambda: bm.expert_order(torch.zeros(4, 2, dtype=torch.int64), 3, stream=1),
                 lambda: bm.expert_gather(torch.zeros(4, 8), _order(), stream=1),
                 lambda: bm.rotary(torch.zeros(4, 2, 8), POS, F, stream=1)):
        with pytest.raises(ValueError, match="device"):
            call()
