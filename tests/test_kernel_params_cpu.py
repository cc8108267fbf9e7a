"""Every member of a kernel's parameter struct is read by the kernel (its file, behind the struct)."""
import os
import re

import pytest

from bit_nf4_quantized_19_b200 import build


def members():
    out = []
    for name in sorted(build.HEADERS):
        text = re.sub(r"//[^\n]*", "", open(os.path.join(build.CSRC, name)).read())
        for m in re.finditer(r"struct (\w*Params) \{(.*?)\n\};", text, re.S):
            out += [(m.group(1), n, text[m.end():]) for n in re.findall(r"[\s*,](\w+)(?:\[\w+\])?\s*(?=[,;])", m.group(2))]
    return out


@pytest.mark.parametrize("struct", sorted({s for s, _, _ in members()}))
def test_every_member_is_read(struct):
    unread = [n for s, n, code in members() if s == struct and not re.search(r"\bp\.%s\b" % n, code)]
    assert not unread
