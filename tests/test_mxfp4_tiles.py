"""The packed-MXFP4 tile kernels as their source has them: what no run on a
GPU can show."""
import os
import re

import pytest
import test_gpu_moe as moe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "post_weight_quantization_autoround_amd", "csrc")


def _code(name):
    """A source without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_stages_are_read_before_the_epilogue_writes_over_them():
    # finish_tile writes where other wavefronts' fragments were.  A barrier alone does not tell that those reads are done:
    # each wavefront has to wait for its own first.
    code = _code("mxfp4_tiles.h")
    assert re.search(r"void lds_written_barrier\(\) \{ asm volatile\(\"s_waitcnt lgkmcnt\(0\)\\n\\ts_barrier\"", code)
    calls = [m.start() for m in re.finditer(r"(?<!void )finish_tile<", code)]
    assert len(calls) == 2
    for at in calls:
        barriers = re.findall(r"\b(\w*barrier)\(\);", code[:at])
        assert barriers[-1] == "lds_written_barrier"


# ---------------------------------------------------- which kernel runs where
class _Rule:
    """A launch function of the sources, evaluated for given sizes: `if`, `else`, blocks, constants of whole numbers and
    quotients of doubles, and launches."""

    def __init__(self, name, function):
        code = _code(name)
        at = code.index("{", code.index(function + "(")) + 1
        depth, end = 1, at
        while depth:
            depth += {"{": 1, "}": -1}.get(code[end], 0)
            end += 1
        self.body = " ".join(code[at:end - 1].split())
        self.launches = set(re.findall(r"(launch_\w+<[^>]*>)\(a, stream\);", self.body))

    def pick(self, **names):
        self.names, self.rest, self.chosen = names, self.body, []
        while self.rest:
            self._statement(True)
        assert len(self.chosen) == 1, self.chosen
        return self.chosen[0]

    def _take(self, pattern):
        m = re.match(pattern, self.rest)
        if m:
            self.rest = self.rest[m.end():].lstrip()
        return m

    def _value(self, text):
        text = re.sub(r"\((\w+) \? (\w+) : (\w+)\)", r"(\2 if \1 else \3)", text)
        text = text.replace(" / (double)", " div ").replace("(double)", "").replace(" / ", " // ").replace(" div ", " / ")
        text = text.replace("&&", " and ").replace("||", " or ").replace("!", " not ").replace("a.", "").replace("(a, ", "(")
        return eval(text, {}, dict(self.names))      # (of this repository's own source)

    def _statement(self, live):
        if self._take(r"return hipGetLastError\(\);"):
            return
        if self._take(r"\{"):
            while not self._take(r"\}"):
                self._statement(live)
            return
        m = self._take(r"const (?:int64_t|double|bool) ([^;]*);")
        if m:
            if "aligned =" not in m[1]:      # (addresses: given)
                for part in re.split(r", (?=\w+ = )", m[1]) if live else []:
                    name, value = part.split(" = ", 1)
                    self.names[name] = self._value(value)
            return
        m = self._take(r"(launch_\w+<[^>]*>)\(a, stream\);")
        if m:
            self.chosen += [m[1]] * live
            return
        assert self._take(r"if "), self.rest[:80]
        end = depth = 0
        for end, c in enumerate(self.rest):
            depth += {"(": 1, ")": -1}.get(c, 0)
            if not depth:
                break
        condition, self.rest = self.rest[:end + 1], self.rest[end + 1:].lstrip()
        yes = bool(live and self._value(condition))
        self._statement(live and yes)
        if self._take(r"else\b"):
            self._statement(live and not yes)


def _up(n, by):
    return -(-n // by)


def _linear_kernel(rule, m, n, k, aligned=True):
    return rule.pick(M=m, N=n, K=k, aligned=aligned and k % 128 == 0 and k >= 256,
                     tiles=lambda bm, bn: _up(m, bm) * _up(n, bn))


def _grouped_kernel(rule, m, e, n, k, aligned=True):
    def likely(bm, bn):
        some = min(e, m)
        return max(m // bm + (some + 1) // 2, some) * _up(n, bn)
    return rule.pick(M=m, E=e, N=n, K=k, aligned=aligned and k % 128 == 0 and k >= 256, likely_tiles=likely)


LINEAR = {"a16": ("mxfp4_tiles.h", "hipError_t launch_a16"), "a4": ("mxfp4_tiles.h", "hipError_t launch_a4")}
GROUPED = {x: (f"mxfp4_grouped_{x}.hip", f"hipError_t launch_mx_grouped_{x}") for x in ("a16", "a4")}

STRIDES = [(1, 40, 288), (3, 101, 288), (16, 4097, 288), (40, 5000, 288), (300, 1003, 288), (300, 9000, 288), (520, 17000, 288)]
ACTIVATED = [(1, 2048, 32), (40, 2048, 64), (300, 9000, 160), (520, 17000, 256)]


def test_the_rule_is_read_as_it_stands():
    rule = _Rule(*LINEAR["a4"])
    assert len(rule.launches) == 9 and len(_Rule(*LINEAR["a16"]).launches) == 9
    assert _linear_kernel(rule, 16, 4096, 32) == "launch_skinny<true>"
    assert _linear_kernel(rule, 17, 4096, 256) == "launch_ring<true, 32, 32, 1, 1, 4, 8, 6>"
    assert _linear_kernel(rule, 512, 11008, 4096) == "launch_a4_tile<128, 256>"
    assert _linear_kernel(rule, 512, 11008, 4096, aligned=False) == "launch_ring<true, 128, 128, 2, 2, 2, 8, 4>"
    assert _linear_kernel(rule, 2048, 11008, 4128) == "launch_ring<true, 256, 256, 2, 4, 1, 4, 4>"
    rule = _Rule(*LINEAR["a16"])
    assert _linear_kernel(rule, 2048, 11008, 4096) == "launch_ring<false, 128, 256, 2, 4, 1, 2, 3, 4>"
    assert _linear_kernel(rule, 8192, 8192, 8192) == "launch_ring<false, 256, 256, 2, 4, 1, 2, 3>"
    rule = _Rule(*GROUPED["a16"])
    assert _grouped_kernel(rule, 4096, 8, 11008, 4096) == "launch_groups<false, 256, 256, 2, 4, 1, 2, 3>"
    assert _grouped_kernel(rule, 96, 64, 2816, 2048) == "launch_groups<false, 32, 128, 1, 4, 1, 4, 4, 2>"


@pytest.mark.parametrize("x", ["a16", "a4"])
def test_gpu_tests_reach_every_kernel(x):
    rule = _Rule(*LINEAR[x])
    for shapes in (moe.SHAPES, STRIDES + moe.STRIDED, ACTIVATED + moe.ACT_SHAPES):
        assert rule.launches == {_linear_kernel(rule, *s) for s in shapes}
    if x == "a4":      # the tile kernels with columns in fours and not
        tiles = {(_linear_kernel(rule, *s), s[1] % 4 == 0) for s in moe.STRIDED}
        assert {(f"launch_a4_tile<{t}>", wide) for t in ("128, 256", "256, 256") for wide in (False, True)} <= tiles
    rule = _Rule(*GROUPED[x])
    assert rule.launches == {_grouped_kernel(rule, mean * e, e, n, k) for mean, e, n, k in moe.ACT_TILED}
    groups = {_grouped_kernel(rule, lead + sum(sizes) + trail, len(sizes), n, k)
              for sizes, lead, trail in moe.GROUPS for n, k in ((33, 96), (300, 288), (1030, 1184))}
    assert rule.launches == groups | {_grouped_kernel(rule, mean * e + 3, e, n, k) for mean, e, n, k in moe.TILED}
