"""Waits between a matrix product and what uses its result, in gfx950 assembly.

A product's result may be read or overwritten by another kind of instruction
only some issued instructions later, which the compiler fills with s_nop.  find()
follows every way on from each product and names the uses that come too early.
"""
import re
import sys

# issued instructions between a product and another use of its result
WAITS = (("16x16x32", 7), ("32x32x16", 11), ("16x16x4_f32", 10), ("32x32x2_f32", 18))


def _registers(text):
    m = re.match(r"^-?\|?([av])(?:(\d+)|\[(\d+):(\d+)\])\|?$", text)
    if not m:
        return frozenset()
    first, last = (m[2], m[2]) if m[2] else (m[3], m[4])
    return frozenset((m[1], i) for i in range(int(first), int(last) + 1))


def _blocks(body):
    """Label -> instructions as (name, operands), in order."""
    blocks, now = {"": []}, ""
    for line in body.splitlines()[1:]:
        line = line.split(";")[0].strip()
        label = re.match(r"^(\.LBB\S+):", line)
        if label:
            now = label[1]
            blocks[now] = []
        elif line and not line.startswith(".") and not line.endswith(":"):
            name, _, rest = line.partition(" ")
            blocks[now].append((name, [t.strip().split(" ")[0] for t in rest.split(",")]))
    return blocks


def _early(blocks, after, label, at, left, result, seen):
    """The first use of `result` within `left` instructions, or None."""
    for name, operands in blocks[label][at:]:
        if left <= 0 or name == "s_endpgm":
            return None
        if name == "s_nop":
            left -= int(operands[0], 0) + 1
            continue
        if name.startswith(("s_branch", "s_cbranch")):
            to = operands[0]
            if to in blocks and (to, left, result) not in seen:
                seen.add((to, left, result))
                found = _early(blocks, after, to, 0, left - 1, result, seen)
                if found:
                    return found
            if name == "s_branch":
                return None
            left -= 1
            continue
        used = [_registers(t) for t in operands]
        if name.startswith("v_mfma"):
            # its third factor is the sum so far, which the unit itself keeps in order
            if (used[1] | used[2]) & result:
                return name, operands
            result -= used[0]
            if not result:
                return None
        elif frozenset().union(*used) & result:
            return name, operands
        left -= 1
    following = after[label]
    if following is None or left <= 0 or (following, left, result) in seen:
        return None
    seen.add((following, left, result))
    return _early(blocks, after, following, 0, left, result, seen)


def find(assembly):
    """(kernel, product, early use) of each product whose result is used too early."""
    sys.setrecursionlimit(max(sys.getrecursionlimit(), 20000))
    found = []
    for body in re.split(r"\n(?=_Z\w+:)", assembly)[1:]:
        kernel, body = body.split(":", 1)[0], body.split(".Lfunc_end")[0]
        blocks = _blocks(body)
        labels = list(blocks)
        after = dict(zip(labels, labels[1:] + [None]))
        for label in labels:
            for i, (name, operands) in enumerate(blocks[label]):
                if not name.startswith("v_mfma"):
                    continue
                wait = [n for form, n in WAITS if form in name]
                assert wait, "no wait known for " + name
                use = _early(blocks, after, label, i + 1, wait[0], _registers(operands[0]), set())
                if use:
                    found.append((kernel, (name, operands), use))
    return found
