"""How the kernels read device memory that an earlier kernel may have written.

Every kernel is a programmatic dependent launch: its CTAs may be resident while
the kernels before it still run, so what those write changes within its
lifetime, and the non-coherent path (__ldg, ld.global.nc) may then give values
from before.  The compiler may also choose that path by itself for a pointer
that is const and __restrict__, so such pointers are read by the coherent load
intrinsics (__ldcg, __ldca) or by TMA, never by a plain dereference."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "combine_moe_route_04_gb300", "csrc")
SOURCES = sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh")))


def code(name):
    with open(os.path.join(CSRC, name), encoding="utf-8") as f:
        text = re.sub(r"/\*.*?\*/", " ", f.read(), flags=re.S)
    return re.sub(r"//[^\n]*", "", text)


def plain_reads(text):
    """Names of const __restrict__ pointers that the function declaring them
    subscripts or dereferences."""
    found = set()
    for function in re.split(r"__global__|__device__", text):
        for n in re.findall(r"const\s+\w+\s*\*\s*__restrict__\s+(\w+)", function):
            if re.search(r"(?<![\w.>])%s\s*\[|[=(,&|!<>+\-?:]\s*\*\s*%s\b" % (n, n), function):
                found.add(n)
    return sorted(found)


def test_the_search_finds_what_it_is_for():
    assert plain_reads("void f(const int* __restrict__ a) { int x = a[3]; }") == ["a"]
    assert plain_reads("void f(const float* __restrict__ p) { float x = *p; }") == ["p"]
    assert plain_reads("void f(const int* __restrict__ a) { int x = __ldcg(a + 3) + s.a[1]; }") == []


@pytest.mark.parametrize("name", SOURCES)
def test_no_read_takes_the_non_coherent_path(name):
    text = code(name)
    assert not re.findall(r"__ldg\s*\(|ld\.global(?:\.\w+)*\.nc\b", text)
    assert plain_reads(text) == []
