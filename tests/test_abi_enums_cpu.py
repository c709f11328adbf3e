"""Every enum of the C ABI has all ints among its values, negative ones too, so
that whatever a caller passes is checked and not undefined: its members reach
both ends of int (compiled with g++), and the header stays plain C."""
import os
import re
import shutil
import subprocess

import pytest

INCLUDE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")


def enums():
    text = open(os.path.join(INCLUDE, "cc.h")).read()
    return [(name, re.search(r"(CC_\w+)_MAX_ENUM", body).group(1))
            for body, name in re.findall(r"typedef enum \{([^}]*)\} (cc_\w+_t);", text)]


def test_enums_reach_both_ends_of_int(tmp_path):
    gxx, gcc = shutil.which("g++"), shutil.which("gcc")
    if gxx is None or gcc is None:
        pytest.skip("gcc is not installed")
    names = enums()
    assert len(names) >= 7 and {"cc_dtype_t", "cc_act_t", "cc_status_t"} <= {n for n, _ in names}
    (tmp_path / "enums.cpp").write_text("#include <type_traits>\n#include <limits.h>\n#include \"cc.h\"\n" + "\n".join(
        f'static_assert(std::is_same<std::underlying_type<{n}>::type, int>::value, "{n}");\n'
        f'static_assert((int){p}_MIN_ENUM == INT_MIN && (int){p}_MAX_ENUM == INT_MAX, "{n}");' for n, p in names))
    (tmp_path / "plain.c").write_text('#include "cc.h"\nint main(void) { return sizeof(cc_dtype_t) != sizeof(int); }\n')
    for cmd in ([gxx, "-std=c++17", "-Wall", "-Werror", "-fsyntax-only", "enums.cpp"],
                [gcc, "-std=c99", "-Wall", "-pedantic-errors", "-fsyntax-only", "plain.c"]):
        r = subprocess.run([*cmd, "-I", INCLUDE], cwd=tmp_path, capture_output=True, text=True, timeout=120)
        assert r.returncode == 0, r.stderr[-2000:]
