"""Every wait of the kernels tells somebody when it runs out, read off the sources."""
import glob
import os
import re

from paged_sparse_attention_gb300 import build


def calls(text, name):
    """Argument lists of the calls of ``name`` (not its definition)."""
    for m in re.finditer(r"(?<![\w:])" + name + r"\(", text):
        if re.search(r"(?:bool|void)\s+$", text[:m.start()]):
            continue
        depth, at, args = 1, m.end(), [""]
        while depth:
            c = text[at]
            depth += (c in "([{") - (c in ")]}")
            if depth == 1 and c == ",":
                args.append("")
            elif depth:
                args[-1] += c
            at += 1
        yield [a.strip() for a in args]


def test_every_wait_has_an_error_word():
    seen = 0
    for path in sorted(glob.glob(os.path.join(build.CSRC, "*.cu*"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for name in ("mbar_wait", "mbar_wait_cluster"):
            for args in calls(text, name):
                seen += 1
                assert len(args) >= 3 and args[2] != "nullptr", (os.path.basename(path), name, args)
    assert seen > 20
