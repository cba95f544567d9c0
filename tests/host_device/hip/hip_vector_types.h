// The vector types that the library's headers name.
#pragma once

struct int4 {
    int x, y, z, w;
};
struct float2 {
    float x, y;
};
